// gdn_quantize_i8.cu -- rows to 8-bit integers with one scale a row, and the
// same with the residual's addition and the RMS norm before it.
//
// Per row (D elements, T = the residual's type):
//   norm:   h = round_T(x + residual)         (x alone without a residual)
//           a = fp32(h * weight)
//           scale = m / (127 sqrt(mean(h^2) + eps)),  m = max |a|
//   plain:  a = x,  scale = m / 127
//   q = 127 a / m to the nearest integer, halves to even.
// The norm's 1/rms is a factor of the whole row, so it drops out of q and
// enters only the scale: one pass gathers the sum of squares and the maximum
// together, and q does not depend on the order in which the squares are
// summed. h is rounded to the residual's type before the norm reads it,
// because that is the row the next layer reads back.
//
// The integers are decided exactly: t = a * fp32(127 / m) is within 1.6e-5 of
// 127 a / m, and where t lies closer than 2^-15 to a half the side is taken
// from the sign of 254 |a| - (2 floor|t| + 1) m, whose two products are exact
// in double. The squares are summed in double: no row of finite values
// overflows, and the scale is rounded to fp32 once.
#include <cuda_bf16.h>

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"

namespace gdn {

namespace {

constexpr int kVec = 8;              // elements a thread moves at once
constexpr int kMaxThreads = 1024;    // threads of a row
constexpr int kMaxGroups = 4;        // groups of kVec a thread keeps in registers

__device__ __forceinline__ void load8(const float* p, float (&v)[kVec]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[kVec]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void round_to(float*, float (&)[kVec]) {}
__device__ __forceinline__ void round_to(__nv_bfloat16*, float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
// (the values are bf16 already: their low halves are zero, or they are NaN)
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kVec]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = __byte_perm(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), 0x7632);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// The row's factors once its maximum is known. Rows whose maximum is below
// 1e-30 are raised by 2^100 first (exactly), so that 127 / m stays finite.
struct RowQuant {
    float up, m, r;
    bool zero;       // nothing to scale, or a value that is not finite: q = 0
    __device__ explicit RowQuant(uint32_t mbits) {
        const float top = __uint_as_float(mbits);
        zero = mbits == 0u || mbits >= 0x7f800000u;
        up = top < 1e-30f ? 0x1p100f : 1.0f;
        m = top * up;
        r = zero ? 0.0f : __fdiv_rn(127.0f, m);
    }
    // 127 a / m to the nearest integer as the low byte.
    __device__ uint32_t operator()(float a0) const {
        constexpr float kMagic = 12582912.0f;       // 1.5 * 2^23: the sum's low bits are rint(t)
        const float a = zero ? 0.0f : a0 * up;
        const float t = __fmul_rn(a, r);
        const float s = __fadd_rn(t, kMagic);
        uint32_t q = __float_as_uint(s);
        if (fabsf(t - __fadd_rn(s, -kMagic)) > 0.5f - 0x1p-15f) {
            const float f = floorf(fabsf(t));
            const double c = 254.0 * static_cast<double>(fabsf(a)) -
                             static_cast<double>(2.0f * f + 1.0f) * static_cast<double>(m);
            const int k = static_cast<int>(f);
            const int n = c > 0.0 ? k + 1 : c < 0.0 ? k : k + (k & 1);
            q = static_cast<uint32_t>(a < 0.0f ? -n : n);
        }
        return q;
    }
    __device__ uint2 pack8(const float (&a)[kVec]) const {
        uint32_t b[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) b[i] = (*this)(a[i]);
        uint2 o;
        o.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        o.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
        return o;
    }
};

__device__ __forceinline__ double warp_sum_f64(double x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
    return x;
}

// One row by blockDim.x threads, blockDim.y rows a block. A thread keeps its
// NG groups of 8 in registers between the two halves of the pass; NG = 0 (rows
// too long for that) reads them again, from the residual it has just written
// where there is one.
template <typename XT, typename RT, bool kNorm, int NG>
__global__ void __launch_bounds__(kMaxThreads)
quantize_rows_kernel(const XT* __restrict__ x, const RT* residual, const float* __restrict__ weight,
                     float eps, RT* residual_out, int8_t* __restrict__ q,
                     float* __restrict__ scale, int M, int64_t D) {
    __shared__ double s_sum[32];
    __shared__ uint32_t s_max[32];
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < M;
    const int64_t base = row * D;
    const int T = blockDim.x;
    const int n_groups = static_cast<int>(D / kVec);

    double sum = 0.0;
    uint32_t top = 0;
    // h of a group from its inputs; the statistics' share of it, leaving a
    auto load = [&](int g, float (&v)[kVec], float (&r)[kVec]) {
        const int64_t at = base + static_cast<int64_t>(g) * kVec;
        load8(x + at, v);
        if (kNorm && residual) load8(residual + at, r);
    };
    auto first = [&](int g, float (&a)[kVec], const float (&r)[kVec]) {
        const int64_t at = static_cast<int64_t>(g) * kVec;
        if constexpr (kNorm) {
            if (residual) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) a[i] = __fadd_rn(a[i], r[i]);
            }
            round_to(static_cast<RT*>(nullptr), a);
            if (residual_out) store8(residual_out + base + at, a);
            float w[kVec];
            load8(weight + at, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                sum = fma(static_cast<double>(a[i]), static_cast<double>(a[i]), sum);
                a[i] = __fmul_rn(a[i], w[i]);
            }
        }
        // as bits, so that a NaN is above everything and stays
#pragma unroll
        for (int i = 0; i < kVec; ++i) top = max(top, __float_as_uint(fabsf(a[i])));
    };
    float keep[NG > 0 ? NG : 1][kVec];
    float res[NG > 0 ? NG : 1][kVec];
    if (live) {
        if constexpr (NG > 0) {
            // every load of the thread before its first store: the residual
            // may be updated in place, so the compiler keeps that order
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int g = threadIdx.x + i * T;
                if (g < n_groups) load(g, keep[i], res[i]);
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int g = threadIdx.x + i * T;
                if (g < n_groups) first(g, keep[i], res[i]);
            }
        } else {
            for (int g = threadIdx.x; g < n_groups; g += T) {
                load(g, keep[0], res[0]);
                first(g, keep[0], res[0]);
            }
        }
    }

    // the row's maximum for every thread, its sum for its first warp
    top = __reduce_max_sync(kFull, top);
    if constexpr (kNorm) sum = warp_sum_f64(sum);
    const int warps = T >> 5;                       // warps of a row
    if (warps > 1) {
        const int w0 = threadIdx.y * warps;
        const int lane = threadIdx.x & 31;
        if (lane == 0) {
            s_max[w0 + (threadIdx.x >> 5)] = top;
            if constexpr (kNorm) s_sum[w0 + (threadIdx.x >> 5)] = sum;
        }
        __syncthreads();
        top = __reduce_max_sync(kFull, lane < warps ? s_max[w0 + lane] : 0u);
        if constexpr (kNorm) {
            if (threadIdx.x < 32) sum = warp_sum_f64(lane < warps ? s_sum[w0 + lane] : 0.0);
        }
    }
    if (!live) return;
    const RowQuant rq(top);
    int8_t* qrow = q + base;
    if constexpr (NG > 0) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int g = threadIdx.x + i * T;
            if (g < n_groups)
                *reinterpret_cast<uint2*>(qrow + static_cast<int64_t>(g) * kVec) = rq.pack8(keep[i]);
        }
    } else {
        for (int g = threadIdx.x; g < n_groups; g += T) {
            const int64_t at = static_cast<int64_t>(g) * kVec;
            float a[kVec];
            if (kNorm && residual_out) {
                load8(residual_out + base + at, a);       // this thread wrote it above
            } else {
                float r[kVec];
                load(g, a, r);
                if (kNorm && residual) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) a[i] = __fadd_rn(a[i], r[i]);
                }
                if constexpr (kNorm) round_to(static_cast<RT*>(nullptr), a);
            }
            if constexpr (kNorm) {
                float w[kVec];
                load8(weight + at, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) a[i] = __fmul_rn(a[i], w[i]);
            }
            *reinterpret_cast<uint2*>(qrow + at) = rq.pack8(a);
        }
    }
    if (threadIdx.x == 0) {
        double s = static_cast<double>(__uint_as_float(top)) / 127.0;
        if constexpr (kNorm)
            s /= sqrt(sum / static_cast<double>(D) + static_cast<double>(eps));
        scale[row] = top == 0u ? 0.0f : top >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                                           : static_cast<float>(s);
    }
}

template <typename XT, typename RT, bool kNorm, int NG>
cudaError_t launch_rows(const RowsI8Args& a, int threads, int rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.M + rows - 1) / rows));
    cfg.blockDim = dim3(static_cast<unsigned>(threads), static_cast<unsigned>(rows));
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<XT, RT, kNorm, NG>,
                              static_cast<const XT*>(a.x), static_cast<const RT*>(a.residual),
                              a.weight, a.eps, static_cast<RT*>(a.residual_out), a.q, a.scale,
                              static_cast<int>(a.M), a.D);
}

template <typename XT, typename RT, bool kNorm>
cudaError_t launch_typed(const RowsI8Args& a, cudaStream_t stream) {
    const int64_t groups = a.D / kVec;
    int64_t ng = (groups + kMaxThreads - 1) / kMaxThreads;
    const int threads = static_cast<int>(std::min<int64_t>(
        kMaxThreads, ((groups + (ng <= 1 ? 1 : ng) - 1) / (ng <= 1 ? 1 : ng) + 31) / 32 * 32));
    const int rows = threads >= 256 ? 1 : 256 / threads;
    if (ng <= 1) return launch_rows<XT, RT, kNorm, 1>(a, threads, rows, stream);
    if (ng <= 2) return launch_rows<XT, RT, kNorm, 2>(a, threads, rows, stream);
    if (ng <= kMaxGroups) return launch_rows<XT, RT, kNorm, kMaxGroups>(a, threads, rows, stream);
    return launch_rows<XT, RT, kNorm, 0>(a, kMaxThreads, 1, stream);
}

}  // namespace

cudaError_t launch_rows_i8(const RowsI8Args& a, cudaStream_t stream) {
    using bf16 = __nv_bfloat16;
    if (a.M == 0) return cudaSuccess;
    if (!a.weight)
        return a.x_bf16 ? launch_typed<bf16, float, false>(a, stream)
                        : launch_typed<float, float, false>(a, stream);
    if (a.x_bf16)
        return a.residual_bf16 ? launch_typed<bf16, bf16, true>(a, stream)
                               : launch_typed<bf16, float, true>(a, stream);
    return a.residual_bf16 ? launch_typed<float, bf16, true>(a, stream)
                           : launch_typed<float, float, true>(a, stream);
}

}  // namespace gdn
