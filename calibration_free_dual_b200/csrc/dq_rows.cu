// dq_rows.cu — row quantization to INT8 with one fp32 scale per row (a token's activations, or an
// output channel's weights): x~ = fl32(X * c), a = max |x~|, d = max(fl32(a / 127), 2^-126),
// q = RNE(fl32(x~ * fl32(1/d))).
//
// A row is read once: the CTA's threads hold it in registers (V chunks of 8 channels each) between
// the maximum and the codes, and the CTA walks down the rows with its column scales in registers
// (c is four bytes a channel, twice a bf16 input's, so reading it per row would triple the L2 traffic)
// and the next row's loads in flight. The maximum is reduced on the bit patterns (non-negative
// floats order as integers, infinities and NaN above every finite value). Rows longer than the registers
// hold are read twice, the second time mostly from L2.
#include <algorithm>

#include "dq_device.cuh"
#include "dq_internal.h"
#include "dq_serve.h"

namespace dq {
namespace {

constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr int CH = 8;                     // channels per chunk (one 16-byte load of bf16)
constexpr int MAX_NT = 512;

template <bool F32IN>
struct Raw8 {
  uint4 u[F32IN ? 2 : 1];
};

template <bool F32IN>
__device__ __forceinline__ Raw8<F32IN> load8(const char* row, int64_t chunk) {
  Raw8<F32IN> r;
  const uint4* p = reinterpret_cast<const uint4*>(row) + chunk * (F32IN ? 2 : 1);
#pragma unroll
  for (int i = 0; i < (F32IN ? 2 : 1); ++i) r.u[i] = __ldg(p + i);
  return r;
}

// x~ of a chunk
template <bool F32IN>
__device__ __forceinline__ void rescale8(const Raw8<F32IN>& r, const float (&c)[CH], float (&x)[CH]) {
  if constexpr (F32IN) {
    const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[1].x, r.u[1].y, r.u[1].z, r.u[1].w};
#pragma unroll
    for (int i = 0; i < CH; ++i) x[i] = __fmul_rn(__uint_as_float(w[i]), c[i]);
  } else {
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_f2(w[i]);
      x[2 * i] = __fmul_rn(f.x, c[2 * i]);
      x[2 * i + 1] = __fmul_rn(f.y, c[2 * i + 1]);
    }
  }
}

__device__ __forceinline__ void load_c8(const float* c, int64_t chunk, bool in, float (&v)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] = 1.0f;
  if (c != nullptr && in) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(c) + 2 * chunk);
    const float4 b = __ldg(reinterpret_cast<const float4*>(c) + 2 * chunk + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <int N>
__device__ __forceinline__ uint32_t absmax_bits(const float (&x)[N]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return a;
}

// The CTA's maximum of `a` (bit patterns); `slots` is used in turn by `parity`, so that one barrier a row
// is enough
__device__ __forceinline__ uint32_t block_max(uint32_t a, uint32_t (*slots)[MAX_NT / 32], int parity) {
  a = __reduce_max_sync(FULL, a);
  const int lane = threadIdx.x & 31, nw = blockDim.x / 32;
  if (lane == 0) slots[parity][threadIdx.x / 32] = a;
  __syncthreads();
  return __reduce_max_sync(FULL, lane < nw ? slots[parity][lane] : 0u);
}

struct RowScale {
  float d, inv;
  bool bad;
};
// |x~| <= a, so |x~ / d| <= 127 (1 + 2^-22): the codes stay within -127..127 without a clamp
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  RowScale s;
  const float a = __uint_as_float(bits);
  s.bad = bits >= 0x7F800000u;
  s.d = fmaxf(div_qmax<127>(a), 0x1p-126f);
  s.inv = __frcp_rn(s.d);
  if (bits == 0u) s.d = s.inv = 0.0f;
  if (s.bad) {
    s.d = __uint_as_float(0x7FC00000u);
    s.inv = 0.0f;
  }
  return s;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[CH], const RowScale& s) {
  // adding 1.5 * 2^23 rounds to the nearest integer (ties to even) and leaves its two's
  // complement in the low byte
  uint32_t b[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i)
    b[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], s.inv), 12582912.0f));
  uint2 w;
  w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  if (s.bad) w.x = w.y = 0u;
  return w;
}

// RD rows of a CTA in flight
template <bool F32IN, int V, int RD>
__global__ void __launch_bounds__(MAX_NT)
row_quant_kernel(const RowsArgs A) {
  // a product launched behind this kernel may start loading its weight
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int Q = F32IN ? 2 : 1;                  // 16-byte pieces of a chunk
  extern __shared__ __align__(16) uint4 ring[];      // [RD][V][Q][threads]
  __shared__ uint32_t slots[2][MAX_NT / 32];
  const int64_t chunks = A.n / CH, step = A.ldx * (F32IN ? 4 : 2);
  const int nt = blockDim.x, tid = threadIdx.x;
  const char* X = static_cast<const char*>(A.X) + (int64_t)tid * CH * (F32IN ? 4 : 2);
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring + tid));
  float c[V][CH];
  bool in[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in[i] = tid + (int64_t)i * nt < chunks;
    load_c8(A.c, tid + (int64_t)i * nt, in[i], c[i]);
  }
  auto fetch = [&](int64_t row, int slot) {
    if (row < A.rows) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (in[i]) {
          const char* src = X + row * step + (int64_t)i * nt * CH * (F32IN ? 4 : 2);
#pragma unroll
          for (int h = 0; h < Q; ++h)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         :: "r"(mine + (uint32_t)(((slot * V + i) * Q + h) * nt) * 16u), "l"(src + 16 * h) : "memory");
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int64_t stride = gridDim.x;
#pragma unroll
  for (int d = 0; d < RD; ++d) fetch(blockIdx.x + d * stride, d);
  int parity = 0, slot = 0;
  bool bad = false;
  for (int64_t row = blockIdx.x; row < A.rows; row += stride, parity ^= 1) {
    asm volatile("cp.async.wait_group %0;" :: "n"(RD - 1) : "memory");
    float x[V][CH];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Raw8<F32IN> r = {};
      if (in[i]) {
#pragma unroll
        for (int h = 0; h < Q; ++h) r.u[h] = ring[((slot * V + i) * Q + h) * nt + tid];
      }
      rescale8<F32IN>(r, c[i], x[i]);
      a = max(a, absmax_bits(x[i]));
    }
    fetch(row + RD * stride, slot);                  // this thread's chunks are in registers
    slot = slot + 1 == RD ? 0 : slot + 1;
    const RowScale s = row_scale(block_max(a, slots, parity));
    bad |= s.bad;
    if (tid == 0) A.scales[row] = s.d;
    uint2* dst = reinterpret_cast<uint2*>(A.codes + row * A.n);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (in[i]) dst[tid + (int64_t)i * nt] = codes8(x[i], s);
  }
  if (bad && tid == 0) atomicOr(A.err_word, ERRBIT_NONFINITE);
}

// rows longer than the registers of one CTA: one pass for the maximum, one for the codes
template <bool F32IN>
__global__ void __launch_bounds__(MAX_NT)
row_quant_long_kernel(const RowsArgs A) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t slots[2][MAX_NT / 32];
  const int64_t chunks = A.n / CH, step = A.ldx * (F32IN ? 4 : 2);
  const char* X = static_cast<const char*>(A.X);
  int parity = 0;
  bool bad = false;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, parity ^= 1) {
    uint32_t a = 0;
    float c[CH], x[CH];
    for (int64_t k = threadIdx.x; k < chunks; k += blockDim.x) {
      load_c8(A.c, k, true, c);
      rescale8<F32IN>(load8<F32IN>(X + row * step, k), c, x);
      a = max(a, absmax_bits(x));
    }
    const RowScale s = row_scale(block_max(a, slots, parity));
    bad |= s.bad;
    if (threadIdx.x == 0) A.scales[row] = s.d;
    uint2* dst = reinterpret_cast<uint2*>(A.codes + row * A.n);
    for (int64_t k = threadIdx.x; k < chunks; k += blockDim.x) {
      load_c8(A.c, k, true, c);
      rescale8<F32IN>(load8<F32IN>(X + row * step, k), c, x);
      dst[k] = codes8(x, s);
    }
  }
  if (bad && threadIdx.x == 0) atomicOr(A.err_word, ERRBIT_NONFINITE);
}

template <bool F32IN, int V>
cudaError_t launch_v(const RowsArgs& A, int nt, cudaStream_t s) {
  constexpr int RD = F32IN && V == 4 ? 2 : 4;
  constexpr auto K = row_quant_kernel<F32IN, V, RD>;
  const int smem = RD * V * nt * CH * (F32IN ? 4 : 2);
  if (smem > 48 * 1024) {                           // (what every kernel may have)
    const cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  // as many CTAs as the SMs hold at a time (threads; registers for the wider ones; shared memory)
  const int64_t hold = std::max(1, std::min(2048 / nt / (V == 4 ? 2 : 1), 224 * 1024 / (smem + 1280)));
  K<<<(unsigned)std::min<int64_t>(A.rows, SERVE_SMS * hold), nt, smem, s>>>(A);
  count_launches(1);
  return cudaGetLastError();
}

template <bool F32IN>
cudaError_t launch_rows(const RowsArgs& A, cudaStream_t s) {
  const int64_t chunks = A.n / CH;
  // few rows: the fewest chunks a thread that fit a CTA, for latency. Rows enough for all SMs: four chunks a
  // thread, so that more and smaller CTAs overlap their barriers (8192 x 4096 bf16: 26.6 us with one
  // chunk a thread, 512 threads).
  int v = chunks <= MAX_NT ? 1 : chunks <= 2 * MAX_NT ? 2 : chunks <= 4 * MAX_NT ? 4 : 0;
  if (v != 0 && A.rows > 4 * SERVE_SMS) v = chunks >= 4 * 64 ? 4 : chunks >= 2 * 64 ? 2 : 1;
  const int nt = v == 0 ? MAX_NT : (int)align_up((size_t)(chunks + v - 1) / v, 32);
  switch (v) {
    case 1: return launch_v<F32IN, 1>(A, nt, s);
    case 2: return launch_v<F32IN, 2>(A, nt, s);
    case 4: return launch_v<F32IN, 4>(A, nt, s);
    default: break;
  }
  row_quant_long_kernel<F32IN><<<(unsigned)std::min<int64_t>(A.rows, 4 * SERVE_SMS), nt, 0, s>>>(A);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_row_quant(const RowsArgs& A, int esize, cudaStream_t s) {
  return esize == 4 ? launch_rows<true>(A, s) : launch_rows<false>(A, s);
}

}  // namespace dq
