// dq_gemm8.cu — product of two INT8 operands with a scale per row of each:
// y[t, i] = fl32(fl32(sum_j x[t, j] w[i, j]) * fl32(xs[t] * ws[i])), the integer sum exact.
//
// sm_100a design: tcgen05.mma.kind::i8 (32 channels per instruction, int32 accumulators in tensor
// memory). The weight rows are the MMA's 128 rows and the tokens its columns, so that few tokens
// make a narrow tile instead of an idle one, and the epilogue's lanes run along a row of y.
//   * warp 0 (one lane): per slice of 128 channels, one TMA tile load of either operand (128-byte
//     swizzle) on the slice's "full" mbarrier;
//   * warp 1: four MMAs per slice, committed to the slice's "empty" mbarrier;
//   * warps 2-5: the accumulator, converted and scaled, to y.
// Every wait is bounded; on timeout the kernel raises the error word, frees its TMEM and returns.
#include <algorithm>
#include <cstring>

#include "dq_device.cuh"
#include "dq_internal.h"
#include "dq_serve.h"
#include "dq_tc.cuh"

namespace dq {
namespace {

constexpr unsigned FULL_MASK = 0xFFFFFFFFu;
constexpr int GT = 192;
constexpr int BM = 128;                 // weight rows of a tile
constexpr int BK = 128;                 // channels (bytes) of a slice

// A, B signed 8-bit, D int32, both operands K-major
__host__ __device__ constexpr uint32_t idesc_i8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected) : "memory");
}

template <int BN>
struct Cfg {
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 128 ? 3 : 5;
  static constexpr int BAR = STAGES * STAGE;
  static constexpr int SMEM = BAR + 256 + 1024;
  static constexpr uint32_t COLS = BN < 32 ? 32 : BN;
};

template <int BN, bool BF16OUT>
__global__ void __launch_bounds__(GT)
gemm8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
             const Gemm8Args A) {
  using C = Cfg<BN>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t n0 = (int64_t)blockIdx.x * BM, t0 = (int64_t)blockIdx.y * BN;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char* base_ptr = smem_raw + (sbase - raw);
  const uint32_t full0 = sbase + C::BAR, empty0 = full0 + 8 * C::STAGES;
  const uint32_t accbar = empty0 + 8 * C::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + C::BAR + 8 * (2 * C::STAGES + 1));
  volatile int* fail = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), C::COLS);
  if (tid == 32) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(accbar, 1);
    *fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nk = (int)((A.K + BK - 1) / BK);

  if (warp == 0 && lane == 0) {
    // the weight does not depend on the quantizer's launch: its first slices go ahead
    const int head = nk < C::STAGES ? nk : C::STAGES;
    for (int k = 0; k < head; ++k) {
      mbar_expect_tx(full0 + 8 * k, C::STAGE);
      tma_load_2d(sbase + k * C::STAGE, &tmW, k * BK, (int)n0, full0 + 8 * k);
    }
    if (A.after_rows) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int k = 0; k < head; ++k)
      tma_load_2d(sbase + k * C::STAGE + C::A_BYTES, &tmX, k * BK, (int)t0, full0 + 8 * k);
    int k = head;
    for (; k < nk; ++k) {
      const int s = k % C::STAGES;
      if (!mbar_wait(empty0 + 8 * s, ((uint32_t)(k / C::STAGES) & 1u) ^ 1u)) { *fail = 1; break; }
      if (*fail) break;
      const uint32_t st = sbase + s * C::STAGE;
      mbar_expect_tx(full0 + 8 * s, C::STAGE);
      tma_load_2d(st, &tmW, k * BK, (int)n0, full0 + 8 * s);
      tma_load_2d(st + C::A_BYTES, &tmX, k * BK, (int)t0, full0 + 8 * s);
    }
    if (*fail)                                     // copies still in flight land before the CTA ends
      for (int j = k > C::STAGES ? k - C::STAGES : 0; j < k; ++j)
        mbar_wait(full0 + 8 * (j % C::STAGES), (uint32_t)(j / C::STAGES) & 1u);
  } else if (warp == 1) {
    const uint32_t elected = elect_lane(), acc = warp_uniform(tmem);
    bool ok = true;
    for (int k = 0; k < nk; ++k) {
      const int s = k % C::STAGES;
      if (!mbar_wait_warp(full0 + 8 * s, (uint32_t)(k / C::STAGES) & 1u) || warp_any(*fail)) {
        *fail = 1;
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = sbase + s * C::STAGE;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb)
        mma_i8(acc, operand_desc(st + 32 * kb), operand_desc(st + C::A_BYTES + 32 * kb),
               idesc_i8(BM, BN), (k > 0 || kb > 0) ? 1u : 0u, elected);
      mma_commit_if(elected, empty0 + 8 * s);
    }
    if (ok) mma_commit_if(elected, accbar);
  } else if (warp >= 2) {
    const int sp = warp & 3;
    const int64_t n = n0 + sp * 32 + lane;
    const float wsc = n < A.N ? __ldg(A.ws + n) : 0.0f;
    if (A.after_rows) asm volatile("griddepcontrol.wait;" ::: "memory");
    int got = 0;
    if (lane == 0) got = (mbar_wait(accbar, 0) && !*fail) ? 1 : 0;
    if (__shfl_sync(FULL_MASK, got, 0)) {
      tc_fence_after();
      const int cols = (int)(A.T - t0 < BN ? A.T - t0 : BN);
#pragma unroll 1
      for (int cb = 0; cb < cols; cb += 32) {
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(sp * 32) << 16) + cb, v);
        const float xsc = cb + lane < cols ? A.xs[t0 + cb + lane] : 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float y = __fmul_rn(__int2float_rn(__float_as_int(v[j])),
                                    __fmul_rn(__shfl_sync(FULL_MASK, xsc, j), wsc));
          if (cb + j < cols && n < A.N) {
            const int64_t at = (t0 + cb + j) * A.ldy + n;
            if (BF16OUT) static_cast<__nv_bfloat16*>(A.y)[at] = __float2bfloat16_rn(y);
            else static_cast<float*>(A.y)[at] = y;
          }
        }
      }
    } else if (lane == 0) {
      *fail = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *fail) atomicOr(A.err_word, ERRBIT_TIMEOUT);
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// [rows, K] bytes, box of box_rows rows x 128 bytes, 128-byte swizzle, zero fill outside
bool codes8_map(CUtensorMap* map, const int8_t* codes, int64_t rows, int64_t K, int box_rows) {
  EncodeTiledFn fn = encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(codes), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool BF16OUT>
cudaError_t launch_tile(const Gemm8Args& A, cudaStream_t s) {
  using C = Cfg<BN>;
  alignas(64) CUtensorMap tw, tx;
  if (!codes8_map(&tw, A.w, A.N, A.K, BM) || !codes8_map(&tx, A.x, A.T, A.K, BN))
    return cudaErrorInvalidValue;
  constexpr auto K = gemm8_kernel<BN, BF16OUT>;
  cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((A.N + BM - 1) / BM), (unsigned)((A.T + BN - 1) / BN));
  cfg.blockDim = dim3(GT);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = A.after_rows ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, K, tw, tx, A);
  count_launches(1);
  return e;
}

template <int BN>
cudaError_t launch_out(const Gemm8Args& A, cudaStream_t s) {
  return A.y_bf16 ? launch_tile<BN, true>(A, s) : launch_tile<BN, false>(A, s);
}

}  // namespace

size_t gemm8_workspace_bytes(int64_t, int64_t, int64_t) { return 16; }

cudaError_t launch_gemm8(const Gemm8Args& A, void*, cudaStream_t s) {
  if (A.T <= 32) return launch_out<32>(A, s);
  return launch_out<128>(A, s);
}

}  // namespace dq
