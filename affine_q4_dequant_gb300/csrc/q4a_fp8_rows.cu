// q4a_fp8_rows.cu -- the bandwidth-bound operators of the 8-bit form:
//   q4a_quantize_fp8     activations to e4m3 with a scale per 128 columns of a row
//   q4a_add_rmsnorm_fp8  the residual's addition and the RMSNorm before that
//   q4a_dequant_fp8      packed 4-bit weights to e4m3 with a scale per 128 x 128 block
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q4a_device.cuh"
#include "q4a_fp8.h"
#include "q4a_internal.h"

namespace q4a {
namespace {

constexpr int kRowElems = 16;   // elements of one thread and chunk: 8 threads share a 128-column block

// 16 consecutive elements as fp32.
__device__ __forceinline__ void load16(const float* p, float (&v)[kRowElems]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = a.x;
        v[4 * i + 1] = a.y;
        v[4 * i + 2] = a.z;
        v[4 * i + 3] = a.w;
    }
}
__device__ __forceinline__ float2 pair_f32(uint32_t w, const __half*) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 pair_f32(uint32_t w, const __nv_bfloat16*) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[kRowElems]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[i];
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = pair_f32(w[k], p);
            v[8 * i + 2 * k] = f.x;
            v[8 * i + 2 * k + 1] = f.y;
        }
    }
}

// v rounded to T, stored, and left in v as the stored value.
__device__ __forceinline__ void store16(float* p, float (&v)[kRowElems], bool write) {
    if (!write) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ uint32_t round_pair(float a, float b, const __half*) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t round_pair(float a, float b, const __nv_bfloat16*) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store16(T* p, float (&v)[kRowElems], bool write) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = 8 * i + 2 * k;
            w[k] = round_pair(v[e], v[e + 1], p);
            const float2 f = pair_f32(w[k], p);
            v[e] = f.x;
            v[e + 1] = f.y;
        }
        if (write) reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Rows to 8 bits. `wpr` warps share a row, thread t of them holding elements 16 t .. 16 t + 15 of
// each of NC chunks in registers, so the row is read once: the sum of squares, the blocks' maxima
// (8 threads a block) and the codes all come from those registers.
template <typename XT, typename RT, bool RES, bool NORM, int NC>
__global__ void __launch_bounds__(NC == 1 ? 1024 : 512)
    fp8_rows_kernel(const Fp8Norm p, int wpr) {
    __shared__ float s_red[32];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5;
    const int rpc = (blockDim.x >> 5) / wpr;                 // rows of this CTA
    const int64_t row = (int64_t)blockIdx.x * rpc + warp / wpr;
    const int t = (int)threadIdx.x - warp / wpr * wpr * 32;  // thread within the row
    const bool live = row < p.nb;
    const int64_t nblk = (p.dim + kFp8Block - 1) / kFp8Block;
    float v[NC][kRowElems];
    float ssq = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t e = ((int64_t)c * wpr * 32 + t) * kRowElems;
        const bool on = live && e < p.dim;
#pragma unroll
        for (int i = 0; i < kRowElems; ++i) v[c][i] = 0.f;
        if (on) {
            load16(static_cast<const XT*>(p.x) + row * p.dim + e, v[c]);
            if (RES) {
                float r[kRowElems];
                load16(static_cast<const RT*>(p.residual) + row * p.dim + e, r);
#pragma unroll
                for (int i = 0; i < kRowElems; ++i) v[c][i] = __fadd_rn(v[c][i], r[i]);
                store16(static_cast<RT*>(p.x_new) + row * p.dim + e, v[c], p.x_new != nullptr);
            }
        }
        if (NORM) {
#pragma unroll
            for (int i = 0; i < kRowElems; ++i) ssq = fmaf(v[c][i], v[c][i], ssq);
        }
    }
    float rstd = 1.f;
    if (NORM) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, o);
        if (wpr > 1) {
            if ((threadIdx.x & 31) == 0) s_red[warp] = ssq;
            __syncthreads();
            const int w0 = warp / wpr * wpr;
            ssq = 0.f;
            for (int w = 0; w < wpr; ++w) ssq += s_red[w0 + w];
        }
        rstd = 1.f / sqrtf(ssq / (float)p.dim + p.eps);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t e = ((int64_t)c * wpr * 32 + t) * kRowElems;
        const bool on = live && e < p.dim;
        if (NORM && on) {
            float w[kRowElems];
            load16(reinterpret_cast<const __nv_bfloat16*>(p.norm_w) + e, w);
#pragma unroll
            for (int i = 0; i < kRowElems; ++i) v[c][i] = v[c][i] * rstd * (w[i] + p.shift);
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < kRowElems; ++i) amax = fmaxf(amax, fabsf(v[c][i]));
#pragma unroll
        for (int o = 1; o < kFp8Block / kRowElems; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (on) {
            const float scale = fp8_scale(amax);
            const float inv = 1.f / scale;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = e4m3x4(v[c][4 * i] * inv, v[c][4 * i + 1] * inv, v[c][4 * i + 2] * inv, v[c][4 * i + 3] * inv);
            *reinterpret_cast<uint4*>(p.q + row * p.dim + e) = make_uint4(o[0], o[1], o[2], o[3]);
            if ((t & (kFp8Block / kRowElems - 1)) == 0) p.scale[row * nblk + e / kFp8Block] = scale;
        }
    }
}

template <typename XT, typename RT, bool RES, bool NORM>
q4a_status launch_rows_typed(const Fp8Norm& n, cudaStream_t stream) {
    // one chunk per thread up to 1024 threads (16384 columns), else four
    const bool wide = n.dim > 1024 * kRowElems;
    const int64_t threads = (n.dim + kRowElems - 1) / kRowElems;
    const int wpr = (int)((wide ? (threads + 127) / 128 : (threads + 31) / 32));
    const int rpc = wpr >= 8 ? 1 : 8 / wpr;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((n.nb + rpc - 1) / rpc), 1, 1);
    cfg.blockDim = dim3((unsigned)(32 * wpr * rpc), 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, fp8_rows_kernel<XT, RT, RES, NORM, 4>, n, wpr)
                               : cudaLaunchKernelEx(&cfg, fp8_rows_kernel<XT, RT, RES, NORM, 1>, n, wpr);
    return e == cudaSuccess ? Q4A_OK : cuda_fail(e);
}

template <typename XT>
q4a_status launch_rows_x(const Fp8Norm& n, cudaStream_t stream) {
    if (!n.norm_w) return launch_rows_typed<XT, float, false, false>(n, stream);
    if (!n.residual) return launch_rows_typed<XT, float, false, true>(n, stream);
    if (n.res_type == Q4A_F32) return launch_rows_typed<XT, float, true, true>(n, stream);
    if (n.res_type == Q4A_F16) return launch_rows_typed<XT, __half, true, true>(n, stream);
    return launch_rows_typed<XT, __nv_bfloat16, true, true>(n, stream);
}

// One CTA per 128 x 128 block, two threads a row, one 64-input group each: W = fma(s, q, b) for the
// block's maximum, then again for the codes.
__global__ void __launch_bounds__(256)
    dequant_fp8_kernel(uint8_t* __restrict__ w8, float* __restrict__ w_scale, const uint8_t* __restrict__ w,
                       const uint16_t* __restrict__ s, const uint16_t* __restrict__ b, int64_t rows, int64_t in_dim) {
    __shared__ float s_max[8];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t nblk = (in_dim + kFp8Block - 1) / kFp8Block;
    const int64_t kb = blockIdx.x % nblk, rb = blockIdx.x / nblk;
    const int64_t row = rb * kFp8Block + (threadIdx.x >> 1);
    const int64_t col = kb * kFp8Block + (threadIdx.x & 1) * kGroup;
    const bool on = row < rows && col < in_dim;
    uint32_t word[8] = {};
    float sv = 0.f, bv = 0.f, amax = 0.f;
    if (on) {
        const uint4* src = reinterpret_cast<const uint4*>(w + row * (in_dim / 2) + col / 2);
        const uint4 a = src[0], c = src[1];
        word[0] = a.x, word[1] = a.y, word[2] = a.z, word[3] = a.w;
        word[4] = c.x, word[5] = c.y, word[6] = c.z, word[7] = c.w;
        sv = bf16_to_f32(s[row * (in_dim / kGroup) + col / kGroup]);
        bv = bf16_to_f32(b[row * (in_dim / kGroup) + col / kGroup]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(fmaf(sv, (float)((word[i] >> (4 * k)) & 15u), bv)));
    }
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = 0.f;
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, s_max[i]);
    const float scale = fp8_scale(amax), inv = 1.f / scale;
    if (threadIdx.x == 0) w_scale[rb * nblk + kb] = scale;
    if (!on) return;
    uint2* dst = reinterpret_cast<uint2*>(w8 + row * in_dim + col);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fmaf(sv, (float)((word[i] >> (4 * k)) & 15u), bv) * inv;
        dst[i] = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
    }
}

}  // namespace

q4a_status launch_fp8_rows(const Fp8Norm& n, cudaStream_t stream) {
    if (n.x_type == Q4A_F32) return launch_rows_x<float>(n, stream);
    if (n.x_type == Q4A_F16) return launch_rows_x<__half>(n, stream);
    return launch_rows_x<__nv_bfloat16>(n, stream);
}

q4a_status launch_dequant_fp8(uint8_t* w8, float* w_scale, const uint8_t* w, const uint16_t* s, const uint16_t* b,
                              int64_t rows, int64_t in_dim, cudaStream_t stream) {
    const int64_t blocks = (rows + kFp8Block - 1) / kFp8Block * ((in_dim + kFp8Block - 1) / kFp8Block);
    if (blocks > ((int64_t)1 << 31) - 1) return Q4A_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, dequant_fp8_kernel, w8, w_scale, w, s, b, rows, in_dim);
    return e == cudaSuccess ? Q4A_OK : cuda_fail(e);
}

}  // namespace q4a
