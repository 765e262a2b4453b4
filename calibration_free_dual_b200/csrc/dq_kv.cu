// dq_kv.cu — new tokens' keys and values into a paged cache, the keys (and the queries) rotated by
// their positions on the way, in bf16 or as INT8 codes with one scale per (token, head).
//
// A memory-bound pass: every value is read once and written once. A head's row belongs to head_dim/8
// threads, each with 8 channels in registers: with the half-split rotation four of the first
// half and their four partners (no exchange between lanes), otherwise 8 in a row. A CTA takes one
// token's rows of all heads, so the token's cos and sin are loaded once a thread. The INT8
// row maximum is reduced by shuffles among the row's threads. 6001 tokens, 32 + 32 + 32 heads of 128, bf16: 52 us,
// 298 MB at 5.7 TB/s (reads and writes mixed); 32 + 8 + 8 heads, INT8 cache: 31 us, 4.5 TB/s (instructions and latency);
// 64 tokens 2.7 us.
#include <algorithm>

#include "dq_device.cuh"
#include "dq_internal.h"
#include "dq_serve.h"

namespace dq {
namespace {

constexpr unsigned FULL = 0xFFFFFFFFu;

// four channels: as they lie in memory, and as binary32
template <bool F32IN>
struct Raw4 {
  uint32_t u[F32IN ? 4 : 2];
};
template <bool F32IN>
__device__ __forceinline__ Raw4<F32IN> load4(const char* p) {
  Raw4<F32IN> r;
  if constexpr (F32IN) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    r.u[0] = v.x; r.u[1] = v.y; r.u[2] = v.z; r.u[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);      // (q may be rotated in place)
    r.u[0] = v.x; r.u[1] = v.y;
  }
  return r;
}
template <bool F32IN>
__device__ __forceinline__ void unpack4(const Raw4<F32IN>& r, float* x) {
  if constexpr (F32IN) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r.u[i]);
  } else {
    const float2 a = bf16x2_to_f2(r.u[0]), b = bf16x2_to_f2(r.u[1]);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
}

__device__ __forceinline__ uint2 pack4(const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

template <int D, bool INT8, bool F32IN, int NT>
__global__ void __launch_bounds__(NT, NT == 64 ? 12 : 1)
kv_append_kernel(const AppendArgs A) {
  constexpr int TPR = D / 8;                        // threads of one head's row
  constexpr int RPP = NT / TPR;                     // rows at a time
  constexpr int ES = F32IN ? 4 : 2;
  const int64_t t = blockIdx.x;
  const int sub = threadIdx.x % TPR;
  const dq_kv_cache& C = A.cache;
  const int G = C.kv_heads, rows = A.q_heads + 2 * G;
  // this thread's channels lo..lo+3 and hi..hi+3 of a rotated row
  const bool halves = A.rot.dim > 0 && !A.rot.interleaved;
  const bool turned = 8 * sub < A.rot.dim;
  const int lo_r = halves && turned ? 4 * sub : 8 * sub;
  const int hi_r = halves && turned ? A.rot.dim / 2 + 4 * sub : 8 * sub + 4;
  // rows of the token: keys, values, queries. The loads of UNR rounds go ahead of their stores, the
  // first ones ahead of the token's slot and position too.
  constexpr int UNR = NT == 64 ? 6 : 4;
  struct { Raw4<F32IN> lo, hi; } x8[UNR];
  const char* kp = static_cast<const char*>(A.k) + t * A.k_stride * ES;
  const char* vp = static_cast<const char*>(A.v) + t * A.v_stride * ES;
  const char* qp = static_cast<const char*>(A.q) + t * A.q_stride * ES;
  const int lane_row = threadIdx.x / TPR;
  auto load_rounds = [&](int first) {
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      const int r = first + u * RPP + lane_row;
      const bool is_q = r >= 2 * G, is_v = !is_q && r >= G;
      const int h = r - (is_q ? 2 * G : is_v ? G : 0);
      const int lo = is_v ? 8 * sub : lo_r, hi = is_v ? 8 * sub + 4 : hi_r;
      x8[u] = {};
      if (r < rows) {
        const char* src = (is_q ? qp : is_v ? vp : kp) + h * (D * ES);
        x8[u].lo = load4<F32IN>(src + lo * ES);
        x8[u].hi = load4<F32IN>(src + hi * ES);
      }
    }
  };
  load_rounds(0);
  const int64_t slot = __ldg(A.slots + t);
  int64_t pos = 0;
  bool ok = slot < C.pages * C.page_size;
  if (A.rot.dim > 0) {
    pos = __ldg(A.rot.positions + t);
    ok = ok && pos >= 0 && pos < A.rot.rows;
  }
  if (!ok) {
    if (threadIdx.x == 0) atomicOr(A.err_word, ERRBIT_BADARG);
    return;
  }
  float cs[4] = {}, sn[4] = {};
  if (turned) {
    unpack4<true>(load4<true>(reinterpret_cast<const char*>(A.rot.cos + pos * (A.rot.dim / 2) + 4 * sub)), cs);
    unpack4<true>(load4<true>(reinterpret_cast<const char*>(A.rot.sin + pos * (A.rot.dim / 2) + 4 * sub)), sn);
  }
  const int lg = __ffs(C.page_size) - 1;
  const int64_t page = slot < 0 ? 0 : slot >> lg, prow = slot < 0 ? 0 : slot & (C.page_size - 1);
  const int64_t at = (page * C.page_stride + prow * C.row_stride) * (INT8 ? 1 : 2);
  char* kdst = static_cast<char*>(C.k) + at;
  char* vdst = static_cast<char*>(C.v) + at;
  char* qo = static_cast<char*>(A.q_out) + t * A.q_out_stride * 2;
  bool bad = false;
  // (whole warps run the same count of rounds)
  for (int first = 0; first < rows; first += UNR * RPP) {
    if (first > 0) load_rounds(first);
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      if (first + u * RPP >= rows) break;
      const int r = first + u * RPP + lane_row;
      const bool is_q = r >= 2 * G, is_v = !is_q && r >= G;
      const bool live = r < rows && (is_q || slot >= 0);
      const int h = r - (is_q ? 2 * G : is_v ? G : 0);
      // a value goes to a bf16 cache as it came
      if (!INT8 && !F32IN && is_v) {
        if (live) {
          char* dst = vdst + h * C.head_stride * 2;
          *reinterpret_cast<uint2*>(dst + 16 * sub) = make_uint2(x8[u].lo.u[0], x8[u].lo.u[1]);
          *reinterpret_cast<uint2*>(dst + 16 * sub + 8) = make_uint2(x8[u].hi.u[0], x8[u].hi.u[1]);
        }
        continue;
      }
      const int lo = is_v ? 8 * sub : lo_r, hi = is_v ? 8 * sub + 4 : hi_r;
      float x[8];
      unpack4<F32IN>(x8[u].lo, x);
      unpack4<F32IN>(x8[u].hi, x + 4);
      if (!is_v && turned) {
        if (halves) {
#pragma unroll
          for (int i = 0; i < 4; ++i) turn(x[i], x[4 + i], cs[i], sn[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
        }
      }
      char* cdst = (is_v ? vdst : kdst) + h * C.head_stride * (INT8 ? 1 : 2);
      if (INT8 && __any_sync(FULL, live && !is_q)) {
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int off = 1; off < TPR; off <<= 1) a = max(a, __shfl_xor_sync(FULL, a, off));
        if (live && !is_q) {
          const bool inf = a >= 0x7F800000u;
          float d = fmaxf(div_qmax<127>(__uint_as_float(a)), 0x1p-126f), inv = __frcp_rn(d);
          if (a == 0u) d = inv = 0.0f;
          if (inf) {
            d = __uint_as_float(0x7FC00000u);
            inv = 0.0f;
            bad = true;
          }
          // (rounding as in the row quantizer: no code leaves -127..127)
          uint32_t b[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            b[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], inv), 12582912.0f));
          uint32_t w0 = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
          uint32_t w1 = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
          if (inf) w0 = w1 = 0u;
          *reinterpret_cast<uint32_t*>(cdst + lo) = w0;
          *reinterpret_cast<uint32_t*>(cdst + hi) = w1;
          if (sub == 0) (is_v ? C.v_scales : C.k_scales)[((page * G + h) << lg) + prow] = d;
        }
      }
      if (live && (!INT8 || is_q)) {
        char* dst = is_q ? qo + h * (D * 2) : cdst;
        *reinterpret_cast<uint2*>(dst + lo * 2) = pack4(x);
        *reinterpret_cast<uint2*>(dst + hi * 2) = pack4(x + 4);
      }
    }
  }
  if (bad) atomicOr(A.err_word, ERRBIT_NONFINITE);
}

template <int D, bool INT8, bool F32IN>
cudaError_t launch_typed(const AppendArgs& A, cudaStream_t s) {
  const unsigned g = (unsigned)A.tokens;
  // Many tokens: 64 threads each, six rounds of loads ahead, so that more tokens are in flight and few threads idle in
  // the last round (6001 tokens, INT8, 32 + 8 + 8 heads: 31 us, with 256 threads 41). Few tokens: 256 threads, for
  // latency (64 tokens of that kind: 2.7 us, with 64 threads 5.0; even at about 600: 6.2 and 6.3), unless
  // 64 threads are done in two rounds anyway (600 tokens, 8 + 2 + 2 heads of 64: 2.9 us, with 256 threads 4.8).
  const bool narrow = A.tokens > 4 * SERVE_SMS || (A.q_heads + 2 * (int64_t)A.cache.kv_heads) * (D / 8) <= 2 * 64;
  if (narrow) kv_append_kernel<D, INT8, F32IN, 64><<<g, 64, 0, s>>>(A);
  else kv_append_kernel<D, INT8, F32IN, 256><<<g, 256, 0, s>>>(A);
  count_launches(1);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const AppendArgs& A, int esize, cudaStream_t s) {
  if (A.cache.kind == DQ_CACHE_INT8)
    return esize == 4 ? launch_typed<D, true, true>(A, s) : launch_typed<D, true, false>(A, s);
  return esize == 4 ? launch_typed<D, false, true>(A, s) : launch_typed<D, false, false>(A, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& A, int esize, cudaStream_t s) {
  return A.cache.head_dim == 64 ? launch_dim<64>(A, esize, s) : launch_dim<128>(A, esize, s);
}

}  // namespace dq
