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

// Packed 4-bit weights to 8-bit blocks. A CTA takes 128 rows x 256 columns (two blocks); a warp 16
// rows, 4 at a time, 8 lanes a row; a lane 32 codes (16 bytes), half of a 64-input group.
//
// Reading 0.56 and writing 1 byte a weight leaves an SM's 128 lanes about 8 instructions a weight at
// the HBM rate, so neither pass works on single weights. W is monotonic in the code (so is the
// rounded multiply-add): a group's largest magnitude is at its smallest or largest code, found on
// pairs of codes where they lie in the packed word. And a group has 16 possible results: its two
// lanes round 8 each to e4m3, and a code becomes its byte by permutes over that table.
constexpr int kDqCols = 256;

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Smallest and largest code of four packed words.
__device__ __forceinline__ void code_range(const uint4& q, uint32_t& lo, uint32_t& hi) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {   // field f of both halves of every word, in place
        const uint32_t m = 0x000F000Fu << (4 * f);
        h[f] = max2(max2(w[0] & m, w[1] & m), max2(w[2] & m, w[3] & m)) >> (4 * f);
        l[f] = min2(min2(w[0] & m, w[1] & m), min2(w[2] & m, w[3] & m)) >> (4 * f);
    }
    const uint32_t a = max2(max2(h[0], h[1]), max2(h[2], h[3])), b = min2(min2(l[0], l[1]), min2(l[2], l[3]));
    hi = max(a & 0xFFFFu, a >> 16);
    lo = min(b & 0xFFFFu, b >> 16);
}

// The bytes of codes 0..3 of a packed half word, from the tables of codes 0..7 (t0, t1) and 8..15
// (t2, t3): a permute takes a byte by three bits, and the fourth chooses between the two.
__device__ __forceinline__ uint32_t table_bytes(uint32_t low3, uint32_t bit3, uint32_t t0, uint32_t t1, uint32_t t2,
                                                uint32_t t3) {
    const uint32_t a = __byte_perm(t0, t1, low3), b = __byte_perm(t2, t3, low3);
    const uint32_t m = __byte_perm(0x0000FF00u, 0u, bit3);
    return (a & ~m) | (b & m);
}

__global__ void __launch_bounds__(256)
    dequant_fp8_kernel(uint8_t* __restrict__ w8, float* __restrict__ w_scale, const uint8_t* __restrict__ w,
                       const uint16_t* __restrict__ s, const uint16_t* __restrict__ b, int64_t rows, int64_t in_dim) {
    __shared__ float s_max[2][8];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t groups = in_dim / kGroup, nblk = (in_dim + kFp8Block - 1) / kFp8Block;
    const int64_t tiles = (in_dim + kDqCols - 1) / kDqCols;
    const int64_t rb = blockIdx.x / tiles, ct = blockIdx.x - rb * tiles;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane & 7;
    const int64_t col = ct * kDqCols + part * 32, row0 = rb * kFp8Block + warp * 16 + (lane >> 3);
    const bool col_on = col < in_dim;
    uint4 q[4];
    uint16_t sb[4], bb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = row0 + 4 * i;
        const bool on = col_on && row < rows;
        q[i] = on ? ld_nc_16(w + row * (in_dim / 2) + col / 2) : make_uint4(0, 0, 0, 0);
        sb[i] = on ? __ldg(s + row * groups + col / kGroup) : (uint16_t)0;
        bb[i] = on ? __ldg(b + row * groups + col / kGroup) : (uint16_t)0;
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        code_range(q[i], lo, hi);
        const float sv = bf16_to_f32(sb[i]), bv = bf16_to_f32(bb[i]);
        amax = fmaxf(amax, fmaxf(fabsf(fmaf(sv, (float)lo, bv)), fabsf(fmaf(sv, (float)hi, bv))));
    }
    // lanes of a block: 4 of a row's 8, in all 4 rows
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
    if (lane == 0) s_max[0][warp] = amax;
    if (lane == 4) s_max[1][warp] = amax;
    __syncthreads();
    const int blk = part >> 2;
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, s_max[blk][i]);
    const float scale = fp8_scale(amax), inv = 1.f / scale;
    if (warp == 0 && (lane == 0 || lane == 4) && col_on) w_scale[rb * nblk + 2 * ct + blk] = scale;
    const float first = (float)((lane & 1) * 8);   // this lane's half of the group's table
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float sv = bf16_to_f32(sb[i]), bv = bf16_to_f32(bb[i]);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fmaf(sv, first + (float)k, bv) * inv;
        const uint32_t m0 = e4m3x4(v[0], v[1], v[2], v[3]), m1 = e4m3x4(v[4], v[5], v[6], v[7]);
        const uint32_t o0 = __shfl_xor_sync(0xffffffffu, m0, 1), o1 = __shfl_xor_sync(0xffffffffu, m1, 1);
        const bool odd = lane & 1;
        const uint32_t t0 = odd ? o0 : m0, t1 = odd ? o1 : m1, t2 = odd ? m0 : o0, t3 = odd ? m1 : o1;
        const uint32_t word[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
        uint32_t out[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t low3 = word[k] & 0x77777777u, bit3 = (word[k] >> 3) & 0x11111111u;
            out[2 * k] = table_bytes(low3, bit3, t0, t1, t2, t3);
            out[2 * k + 1] = table_bytes(low3 >> 16, bit3 >> 16, t0, t1, t2, t3);
        }
        const int64_t row = row0 + 4 * i;
        if (col_on && row < rows) {
            uint4* dst = reinterpret_cast<uint4*>(w8 + row * in_dim + col);
            dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
            dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
        }
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
    const int64_t blocks = (rows + kFp8Block - 1) / kFp8Block * ((in_dim + kDqCols - 1) / kDqCols);
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
