// q4a_fp8_gemm.cu -- the block-scaled 8-bit product and its gated form:
//     y[r][o] = sum_k xs[r][k] ws[o/128][k] sum_{i in block k} x[r][i] w[o][i]
// A plain tiled kernel on the CUDA cores: 16 activation rows x 128 outputs a CTA.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "q4a_device.cuh"
#include "q4a_fp8.h"
#include "q4a_internal.h"

namespace q4a {
namespace {

constexpr int kSimpleRows = 16;   // activation rows of a CTA
constexpr int kSimpleK = 32;      // columns staged at a time

__device__ __forceinline__ float e4m3_f32(uint8_t v) {
    __nv_fp8_e4m3 f;
    f.__x = v;
    return (float)f;
}

// acc[j] = (W x) of activation row row0 + (tid >> 7) * 8 + j and weight row w_row0 + (tid & 127),
// for weight rows below w_rows.
__device__ void product_tile(const Fp8Gemm& p, int64_t row0, int64_t w_row0, int64_t w_rows, float (&acc)[8]) {
    __shared__ float s_w[kFp8Block][kSimpleK + 1];
    __shared__ float s_x[kSimpleRows][kSimpleK + 1];
    const int64_t nblk = (p.in_dim + kFp8Block - 1) / kFp8Block;
    const int col = threadIdx.x & 127, half = threadIdx.x >> 7;
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    for (int64_t kb = 0; kb < nblk; ++kb) {
        float part[8] = {};
        for (int64_t k0 = kb * kFp8Block; k0 < (kb + 1) * kFp8Block && k0 < p.in_dim; k0 += kSimpleK) {
            __syncthreads();
            for (int i = threadIdx.x; i < kFp8Block * kSimpleK; i += 256) {
                const int64_t r = w_row0 + i / kSimpleK, k = k0 + i % kSimpleK;
                s_w[i / kSimpleK][i % kSimpleK] = r < w_rows && k < p.in_dim ? e4m3_f32(p.w[r * p.in_dim + k]) : 0.f;
            }
            for (int i = threadIdx.x; i < kSimpleRows * kSimpleK; i += 256) {
                const int64_t r = row0 + i / kSimpleK, k = k0 + i % kSimpleK;
                s_x[i / kSimpleK][i % kSimpleK] = r < p.nb && k < p.in_dim ? e4m3_f32(p.x[r * p.in_dim + k]) : 0.f;
            }
            __syncthreads();
            for (int k = 0; k < kSimpleK; ++k)
                for (int j = 0; j < 8; ++j) part[j] = fmaf(s_w[col][k], s_x[half * 8 + j][k], part[j]);
        }
        const float ws = w_row0 < w_rows ? p.w_scale[w_row0 / kFp8Block * nblk + kb] : 0.f;
        for (int j = 0; j < 8; ++j) {
            const int64_t r = row0 + half * 8 + j;
            if (r < p.nb) acc[j] = fmaf(part[j], p.x_scale[r * nblk + kb] * ws, acc[j]);
        }
    }
}

__global__ void __launch_bounds__(256) gemm_fp8_kernel(const Fp8Gemm p) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t nt = (p.nb + kSimpleRows - 1) / kSimpleRows;
    const int64_t row0 = blockIdx.x % nt * kSimpleRows, o0 = blockIdx.x / nt * kFp8Block;
    const int col = threadIdx.x & 127, half = threadIdx.x >> 7;
    float acc[8];
    product_tile(p, row0, o0, p.out_dim, acc);
    for (int j = 0; j < 8; ++j) {
        const int64_t r = row0 + half * 8 + j, at = r * p.out_dim + o0 + col;
        if (r >= p.nb || o0 + col >= p.out_dim) continue;
        if (p.y_type == Q4A_F32) static_cast<float*>(p.y)[at] = acc[j];
        else if (p.y_type == Q4A_F16) static_cast<__half*>(p.y)[at] = __float2half_rn(acc[j]);
        else static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(acc[j]);
    }
}

__global__ void __launch_bounds__(256) gate_up_fp8_kernel(const Fp8Gemm p) {
    __shared__ float s_max[8][8];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t nt = (p.nb + kSimpleRows - 1) / kSimpleRows;
    const int64_t row0 = blockIdx.x % nt * kSimpleRows, o0 = blockIdx.x / nt * kFp8Block;
    const int col = threadIdx.x & 127, half = threadIdx.x >> 7;
    float g[8], u[8];
    product_tile(p, row0, o0, 2 * p.out_dim, g);
    product_tile(p, row0, p.out_dim + o0, 2 * p.out_dim, u);
    for (int j = 0; j < 8; ++j) {
        g[j] = g[j] / (1.f + expf(-g[j])) * u[j];
        float m = fabsf(g[j]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5][j] = m;
    }
    __syncthreads();
    for (int j = 0; j < 8; ++j) {
        const int64_t r = row0 + half * 8 + j;
        float m = 0.f;
        for (int i = 0; i < 4; ++i) m = fmaxf(m, s_max[half * 4 + i][j]);
        const float scale = fp8_scale(m), inv = 1.f / scale;
        if (r >= p.nb) continue;
        p.q[r * p.out_dim + o0 + col] = (uint8_t)e4m3x2(g[j] * inv, 0.f);
        if (col == 0) p.scale[r * (p.out_dim / kFp8Block) + o0 / kFp8Block] = scale;
    }
}

}  // namespace

q4a_status launch_gemm_fp8(const Fp8Gemm& g, cudaStream_t stream) {
    const int64_t tiles = (g.nb + kSimpleRows - 1) / kSimpleRows * ((g.out_dim + kFp8Block - 1) / kFp8Block);
    if (tiles > ((int64_t)1 << 31) - 1) return Q4A_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)tiles, 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = g.q ? cudaLaunchKernelEx(&cfg, gate_up_fp8_kernel, g)
                              : cudaLaunchKernelEx(&cfg, gemm_fp8_kernel, g);
    return e == cudaSuccess ? Q4A_OK : cuda_fail(e);
}

}  // namespace q4a
