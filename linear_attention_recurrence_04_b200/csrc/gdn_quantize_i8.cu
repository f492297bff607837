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
// The integers are decided exactly: a * fp32(127 / m) is within 2^-17 of
// 127 a / m, and where it lies closer than 2^-16 to a half the side is taken
// from the sign of 254 |a| - (2 floor|t| + 1) m, whose two products are exact
// in double. The squares are summed in double: no row of finite values
// overflows, and the scale is rounded to fp32 once.
//
// Bound by HBM for many rows: 16384 x 2048 fp32 with an fp32 residual in 64.6 us,
// 16384 x 4096 fp32 quantised in 49.6. (Of the 436 and 336 MB that these move
// 395 and 318 cross the DRAM pins before the kernel ends, 6.0 and 6.4 TB/s of the
// 6.46 of a copy; the last of the writes are still in the L2 then.) bf16 rows,
// with half the bytes for the same instructions, are bound by issue: 40.1 us for
// 16384 x 2048 with a bf16 residual, 10.7 us for 8192 x 2048 quantised, some 2 us
// of that the launch's start and end. Few rows are bound by latency: one row of
// 2048 takes 1.9 us. Rows fetched ahead by persistent blocks (the next row's loads
// in registers) were slower, for want of registers: by 2 % quantising and 40 %
// with the norm for the two bf16 shapes.
#include <cuda_bf16.h>

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"

namespace gdn {

namespace {

constexpr int kVec = 8;              // elements a thread moves at once

// Eight elements as they come from memory.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void unpack(float (&f)[kVec]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[4 * i] = __uint_as_float(v[i].x);
                f[4 * i + 1] = __uint_as_float(v[i].y);
                f[4 * i + 2] = __uint_as_float(v[i].z);
                f[4 * i + 3] = __uint_as_float(v[i].w);
            }
        } else {
            const uint32_t u[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        }
    }
};
__device__ __forceinline__ void round_to(float*, float (&)[kVec]) {}
__device__ __forceinline__ void round_to(__nv_bfloat16*, float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[i], v[i + 1]);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
        v[i] = __uint_as_float(u << 16);
        v[i + 1] = __uint_as_float(u & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
// (the values are bf16 already: their low halves are zero)
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kVec]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = __byte_perm(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), 0x7632);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// max(top, |a|, |b|), a NaN once any of them is one.
__device__ __forceinline__ float max_abs(float top, float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(top), "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// Distances from an integer above this are decided exactly.
constexpr float kNear = 0.5f - 0x1p-16f;
constexpr float kMagic = 12582912.0f;           // 1.5 * 2^23: a sum's low bits are rint

// Two fp32 values in a 64-bit register and the packed operations on them: each
// an issue slot for both. bf16 rows are bound by issue (6 % less time for
// 30000 x 1024); for the fp32 norm the registers that they pair cost more (6 %
// more time for 16384 x 2048).
struct F2 {
    uint64_t v;
    __device__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ explicit F2(uint64_t u) : v(u) {}
    __device__ void get(float& a, float& b) const {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    }
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
    return F2(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
    return F2(r);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.v), "l"(b.v), "l"(c.v));
    return F2(r);
}

__device__ __forceinline__ uint2 low_bytes(const uint32_t (&b)[kVec]) {
    uint2 o;
    o.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return o;
}

// Eight integers of a row of bf16 values, ri = fp32(1 / m), with no case left
// over. Halves are common here (254 a = (2 k + 1) m for one value in a few
// hundred, 8-bit mantissas), so the quotient itself is corrected: p = 127 a
// has 15 bits, the remainder e = p - t m of its first value is exact, and
// t + e ri is then off by less than 2^-24 of it. A quotient that is no half
// is further than 2^-17 of it from one (254 a and (2 k + 1) m differ by a
// unit of the 16 bits they have), and a half is hit exactly.
__device__ __forceinline__ uint2 quantize8_bf16(const float (&a)[kVec], float m, float ri) {
    uint32_t b[kVec];
    const F2 minus_m(-m, -m), ri2(ri, ri), c127(127.0f, 127.0f), magic(kMagic, kMagic);
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
        const F2 p = mul2(F2(a[i], a[i + 1]), c127);
        const F2 t = mul2(p, ri2);
        float s0, s1;
        add2(fma2(fma2(t, minus_m, p), ri2, t), magic).get(s0, s1);
        b[i] = __float_as_uint(s0);
        b[i + 1] = __float_as_uint(s1);
    }
    return low_bytes(b);
}

// Eight integers of any row, r = fp32(127 / m): a r differs from 127 a / m by
// less than 2^-17. `far` grows to the largest distance of an a r from its
// integer.
__device__ __forceinline__ uint2 quantize8(const float (&a)[kVec], float r, float& far) {
    uint32_t b[kVec];
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
        float d[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float s = __fmaf_rn(a[i + j], r, kMagic);
            b[i + j] = __float_as_uint(s);
            d[j] = __fmaf_rn(a[i + j], r, kMagic - s);
        }
        far = max_abs(far, d[0], d[1]);
    }
    return low_bytes(b);
}

// Writes those of eight integers that lie next to a half, on the side that the
// sign of 254 |a| - (2 floor|t| + 1) m gives (both products exact in double).
__device__ __noinline__ void decide8(float a0, float a1, float a2, float a3, float a4, float a5,
                                     float a6, float a7, float m, float r, int8_t* q) {
    const float a[kVec] = {a0, a1, a2, a3, a4, a5, a6, a7};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const float s = __fmaf_rn(a[i], r, kMagic);
        if (fabsf(__fmaf_rn(a[i], r, kMagic - s)) <= kNear) continue;
        const float f = floorf(fabsf(__fmul_rn(a[i], r)));
        const double c = 254.0 * static_cast<double>(fabsf(a[i])) -
                         static_cast<double>(2.0f * f + 1.0f) * static_cast<double>(m);
        const int k = static_cast<int>(f);
        const int n = c > 0.0 ? k + 1 : c < 0.0 ? k : k + (k & 1);
        q[i] = static_cast<int8_t>(a[i] < 0.0f ? -n : n);
    }
}

// Rows whose maximum is not in [kLow, kHigh] are scaled by 2^100 first
// (exactly where it matters), so that 127 / m and 127 a stay finite; rows of
// zeros, and those with a value that is not finite, give zeros.
constexpr float kLow = 1e-30f, kHigh = 1e36f;
__device__ __noinline__ void rare8(float a0, float a1, float a2, float a3, float a4, float a5,
                                   float a6, float a7, uint32_t mbits, int8_t* q) {
    if (mbits == 0u || mbits >= 0x7f800000u) {
        *reinterpret_cast<uint2*>(q) = make_uint2(0, 0);
        return;
    }
    const float up = __uint_as_float(mbits) < kLow ? 0x1p100f : 0x1p-100f;
    const float a[kVec] = {a0 * up, a1 * up, a2 * up, a3 * up, a4 * up, a5 * up, a6 * up, a7 * up};
    const float m = __uint_as_float(mbits) * up, r = __fdiv_rn(127.0f, m);
    float far = 0.0f;
    *reinterpret_cast<uint2*>(q) = quantize8(a, r, far);
    decide8(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], m, r, q);
}

__device__ __forceinline__ double warp_sum_f64(double x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
    return x;
}

// One row by blockDim.x threads, blockDim.y rows a block. A thread keeps its
// NG groups of 8 in registers between the two halves of the pass; NG = 0 (rows
// too long for that) reads them again, from the residual it has just written
// where there is one.
//
// NG depends on the number of rows, and a row's scale must not: the squares are
// summed in an order of the row's own, by 8, then over blocks of 32 groups, then
// over the blocks. So a warp holds NG whole blocks and sums each by itself (rows
// read twice are summed by thread, for every number of rows).
constexpr int max_threads(int ng) { return ng == 4 || ng == 8 ? 512 : 1024; }
// Blocks of that many threads that have to fit an SM: two where fewer registers
// than the compiler would take are faster (bf16 norm of 300 x 8192 in 6.3
// against 8.0 us and of 4096 x 8192 in 41.4 against 43.3; rows read twice,
// 5000 x 36000 bf16 quantised in 115 against 161, but their norm, which spills,
// in 92 against 42 for 100 x 131056 fp32; 8192 x 2048 bf16 quantised with four
// groups 11.0 against 10.3).
constexpr int min_blocks(bool norm, int ng) { return ng == 1 || ng == (norm ? 4 : 0) ? 2 : 1; }

template <typename XT, typename RT, bool kNorm, int NG>
__global__ void __launch_bounds__(max_threads(NG), min_blocks(kNorm, NG))
quantize_rows_kernel(const XT* x, const RT* residual, const float* weight, float eps,
                     RT* residual_out, int8_t* __restrict__ q,
                     float* __restrict__ scale, int M, int64_t D) {
    constexpr int kSums = kNorm && NG > 1 ? NG : 1;  // blocks of 32 groups a warp
    __shared__ double s_sum[max_threads(NG) / 32 * kSums];
    __shared__ uint32_t s_max[32];
    tc::grid_dep_launch();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < M;
    const int64_t base = row * D;
    const int T = blockDim.x;
    const int n_groups = static_cast<int>(D / kVec);
    const int warp = threadIdx.x >> 5;              // of the row
    const int g0 = warp * (32 * NG) + (threadIdx.x & 31);   // the thread's groups: every 32nd
    tc::grid_dep_wait();

    double sums[kSums] = {};
    float top = 0.0f;
    // a of a group from its inputs, with its share of the statistics; the new
    // residual is written
    auto first = [&](int g, const Raw<XT>& xr, const Raw<RT>& rr, const Raw<float>& wr,
                     double& sum, float (&a)[kVec]) {
        const int64_t at = static_cast<int64_t>(g) * kVec;
        xr.unpack(a);
        if constexpr (kNorm) {
            if (residual) {
                float r[kVec];
                rr.unpack(r);
#pragma unroll
                for (int i = 0; i < kVec; ++i) a[i] = __fadd_rn(a[i], r[i]);
            }
            round_to(static_cast<RT*>(nullptr), a);
            if (residual_out) store8(residual_out + base + at, a);
            float w[kVec];
            wr.unpack(w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                sum = fma(static_cast<double>(a[i]), static_cast<double>(a[i]), sum);
                a[i] = __fmul_rn(a[i], w[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kVec; i += 2) top = max_abs(top, a[i], a[i + 1]);
    };
    // The residual may be updated in place: a group is read before it is
    // written. And plain loads do not pass a store that may alias them, so that
    // loads stand before the stores that they need not wait for.
    auto load_x = [&](int g, Raw<XT>& xr, Raw<RT>& rr) {
        const int64_t at = base + static_cast<int64_t>(g) * kVec;
        xr.load(x + at);
        if (kNorm && residual) rr.load(residual + at);
    };
    auto load_w = [&](int g, Raw<float>& wr) {
        if constexpr (kNorm) wr.load(weight + static_cast<int64_t>(g) * kVec);
    };
    float keep[NG > 0 ? NG : 1][kVec];
    if (live) {
        Raw<float> wr;
        if constexpr (NG > 0) {
            Raw<XT> xr[NG];
            Raw<RT> rr[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int g = g0 + 32 * i;
                if (g < n_groups) load_x(g, xr[i], rr[i]);
            }
            // the next group's weights before this one's store where there are
            // registers for both (4096 x 8192 fp32 in 66 us; with four groups
            // the loads before their own store: 16384 x 2048 bf16 in 40.1
            // against 41.4)
            constexpr bool kAhead = NG <= 2;
            Raw<float> wn;
            if (g0 < n_groups) load_w(g0, wr);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int g = g0 + 32 * i;
                if (kAhead && i + 1 < NG && g + 32 < n_groups) load_w(g + 32, wn);
                if (!kAhead && i > 0 && g < n_groups) load_w(g, wr);
                if (g < n_groups) first(g, xr[i], rr[i], wr, sums[kSums > 1 ? i : 0], keep[i]);
                if (kAhead) wr = wn;
            }
        } else {
            // (the next group's loads ahead of this one's arithmetic: 104 us
            // against 87 for 500 x 65536 fp32)
            Raw<XT> xr;
            Raw<RT> rr;
            for (int g = threadIdx.x; g < n_groups; g += T) {
                load_x(g, xr, rr);
                load_w(g, wr);
                first(g, xr, rr, wr, sums[0], keep[0]);
            }
        }
    }

    // the row's maximum for every thread, its sum for its first warp; compared
    // as bits, where infinities and NaN are above everything
    uint32_t mbits = __float_as_uint(top);
    double sum = sums[0];
    const int lane = threadIdx.x & 31;
    if (T < 32) {                                   // several rows a warp, T a power of two
        for (int off = T >> 1; off > 0; off >>= 1) {
            mbits = max(mbits, __shfl_xor_sync(kFull, mbits, off));
            if constexpr (kNorm) sum += __shfl_xor_sync(kFull, sum, off);
        }
    } else {
        mbits = __reduce_max_sync(kFull, mbits);
        if constexpr (kNorm) sum = warp_sum_many<kSums>(sums, lane);
    }
    const int warps = T >> 5;                       // warps of a row
    if (warps > 1 || kSums > 1) {
        const int w0 = threadIdx.y * warps;
        if (lane == 0) s_max[w0 + warp] = mbits;
        if constexpr (kNorm) {
            if (lane % (32 / kSums) == 0)
                s_sum[(w0 + warp) * kSums + lane / (32 / kSums)] = sum;
        }
        __syncthreads();
        mbits = __reduce_max_sync(kFull, lane < warps ? s_max[w0 + lane] : 0u);
        if constexpr (kNorm) {
            if (warp == 0) {
                sum = 0.0;
                for (int b = lane; b < warps * kSums; b += 32) sum += s_sum[w0 * kSums + b];
                sum = warp_sum_f64(sum);
            }
        }
    }
    if (!live) return;
    const float m = __uint_as_float(mbits);
    const bool plain = m >= kLow && m <= kHigh;                 // of the whole row
    constexpr bool kShort = sizeof(XT) == 2 && !kNorm;           // a is bf16
    const float r = __fdiv_rn(kShort ? 1.0f : 127.0f, m);
    int8_t* qrow = q + base;
    auto group = [&](int g) { return qrow + static_cast<int64_t>(g) * kVec; };
    auto exact = [&](int g, const float (&a)[kVec]) {
        decide8(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], m, r, group(g));
    };
    auto rare = [&](int g, const float (&a)[kVec]) {
        rare8(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], mbits, group(g));
    };
    if constexpr (NG > 0) {
        // one test for all of the thread's integers: next to a half lies one
        // in 32768
        float far = 0.0f;
        if (plain) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int g = g0 + 32 * i;
                if (g < n_groups)
                    *reinterpret_cast<uint2*>(group(g)) =
                        kShort ? quantize8_bf16(keep[i], m, r) : quantize8(keep[i], r, far);
            }
        }
        if (!plain || far > kNear) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int g = g0 + 32 * i;
                if (g < n_groups) {
                    if (plain) exact(g, keep[i]);
                    else rare(g, keep[i]);
                }
            }
        }
    } else {
        for (int g = threadIdx.x; g < n_groups; g += T) {
            Raw<XT> xr;
            Raw<RT> rr;
            Raw<float> wr;
            // h as this thread wrote it above, or from its parts
            if (kNorm && residual_out) rr.load(residual_out + base + static_cast<int64_t>(g) * kVec);
            else load_x(g, xr, rr);
            load_w(g, wr);
            float a[kVec];
            if (kNorm && residual_out) {
                rr.unpack(a);
            } else {
                xr.unpack(a);
                if (kNorm && residual) {
                    float f[kVec];
                    rr.unpack(f);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) a[i] = __fadd_rn(a[i], f[i]);
                }
                if constexpr (kNorm) round_to(static_cast<RT*>(nullptr), a);
            }
            if constexpr (kNorm) {
                float w[kVec];
                wr.unpack(w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) a[i] = __fmul_rn(a[i], w[i]);
            }
            if (plain) {
                float far = 0.0f;
                *reinterpret_cast<uint2*>(group(g)) =
                    kShort ? quantize8_bf16(a, m, r) : quantize8(a, r, far);
                if (far > kNear) exact(g, a);
            } else {
                rare(g, a);
            }
        }
    }
    if (threadIdx.x == 0) {
        float s;
        if constexpr (kNorm)
            s = static_cast<float>(static_cast<double>(m) /
                                   (127.0 * sqrt(sum / static_cast<double>(D) +
                                                 static_cast<double>(eps))));
        else
            s = __fdiv_rn(m, 127.0f);
        scale[row] = mbits == 0u ? 0.0f : mbits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : s;
    }
}

template <typename XT, typename RT, bool kNorm, int NG>
cudaError_t launch_rows(const RowsI8Args& a, cudaStream_t stream) {
    const int64_t groups = a.D / kVec;
    int threads = max_threads(0);
    if constexpr (NG > 0) {
        const int64_t need = (groups + NG - 1) / NG;
        threads = 2;
        while (threads < 32 && threads < need) threads *= 2;
        if (need > 32) threads = static_cast<int>((need + 31) / 32 * 32);
    }
    const int rows = threads >= 128 ? 1 : 128 / threads;
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

// Groups a thread. Few rows: one, so that a row is spread over as many threads
// as there are (norm of 64 x 2048 in 2.2 us against 2.5 with two and 4.5 with
// four, of 1000 x 2048 bf16 4.7 against 5.0 and 7.2). Many rows (a million
// threads with one group each, some three waves): as many as put 64 to 128 bytes
// a thread on their way, since what a row costs beside its elements is shared by
// fewer threads (4096 x 8192 bf16 quantised: 20.4 with four, 30.3 with one; bf16
// norm 41.1 against 49.9; fp32 norm 65.6 with two, 67.3 with one and 88 with
// four, which is left out).
// Where the limit is not the best choice: bf16 norm of 4096 x 2048 takes 15.0
// with four and 13.1 with one; quantising rows of middle length below a million
// groups is faster with two (1000 x 6000 bf16 7.3 against 5.5, fp32 8.7 against
// 7.4; 1024 x 4096 fp32 5.5 against 5.4), and 16384 x 512 fp32 with four (8.2
// against 6.0).
template <typename XT, typename RT, bool kNorm>
int groups_a_thread(int64_t M, int64_t groups) {
    const int least = groups <= 1024 ? 1 : groups <= 2048 ? 2 : groups <= 4096 ? 8 : 0;
    if (least != 1 && least != 2) return least;
    if (M * groups < (1 << 20)) return least;
    if (kNorm && sizeof(XT) + sizeof(RT) > 4) return groups > 512 ? 2 : 1;
    if (kNorm) return groups >= 256 ? 4 : 1;
    return groups >= 128 ? 4 : groups >= 64 ? 2 : 1;
}

template <typename XT, typename RT, bool kNorm>
cudaError_t launch_typed(const RowsI8Args& a, cudaStream_t stream) {
    const int64_t groups = a.D / kVec;
    const int ng = groups_a_thread<XT, RT, kNorm>(a.M, groups);
    switch (ng) {
        case 1: return launch_rows<XT, RT, kNorm, 1>(a, stream);
        case 2: return launch_rows<XT, RT, kNorm, 2>(a, stream);
        case 4:
            if constexpr (!kNorm || sizeof(XT) + sizeof(RT) == 4)
                return launch_rows<XT, RT, kNorm, 4>(a, stream);
            return cudaErrorInvalidValue;             // (never chosen for fp32 norms)
        case 8: return launch_rows<XT, RT, kNorm, 8>(a, stream);
        default: return launch_rows<XT, RT, kNorm, 0>(a, stream);
    }
}

// The layer's gated RMS norm (per value head, times norm_w and SiLU(z)) with
// the whole position's row in 8-bit integers: sixteen threads a head, eight
// elements a thread, a block a position. kKeep: every element of the row has
// its thread (at most 64 heads); else the row is formed twice, once for its
// maximum and once for its integers.
template <bool kKeep>
__global__ void __launch_bounds__(1024)
gated_norm_i8_kernel(const float* o, const float* z, const float* norm_w, float eps,
                     int8_t* __restrict__ q, float* __restrict__ scale, int n_groups) {
    __shared__ uint32_t s_max[32];
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    const int T = blockDim.x;                       // a multiple of 32
    const int64_t base = static_cast<int64_t>(blockIdx.x) * n_groups * kVec;
    const int col = static_cast<int>(threadIdx.x % 16) * kVec;
    float w[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = norm_w[col + i];
    // y of a group (zeros past the row: every lane takes part in the sums)
    auto form = [&](int g, float (&y)[kVec]) {
        Raw<float> orr, zrr;
        float zv[kVec];
        const int64_t at = base + static_cast<int64_t>(g < n_groups ? g : 0) * kVec;
        orr.load(o + at);
        zrr.load(z + at);
        orr.unpack(y);
        zrr.unpack(zv);
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            ss = fma(static_cast<double>(y[i]), static_cast<double>(y[i]), ss);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(kFull, ss, off);
        const float inv = static_cast<float>(
            1.0 / sqrt(ss / static_cast<double>(kDv) + static_cast<double>(eps)));
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            y[i] = g < n_groups ? y[i] * inv * w[i] * siluf_acc(zv[i]) : 0.0f;
    };
    float y[kVec];
    float top = 0.0f;
    for (int g0 = 0; g0 < n_groups; g0 += T) {
        form(g0 + threadIdx.x, y);
#pragma unroll
        for (int i = 0; i < kVec; i += 2) top = max_abs(top, y[i], y[i + 1]);
    }
    uint32_t mbits = __reduce_max_sync(kFull, __float_as_uint(top));
    const int lane = threadIdx.x & 31;
    if (lane == 0) s_max[threadIdx.x >> 5] = mbits;
    __syncthreads();
    mbits = __reduce_max_sync(kFull, lane < (T >> 5) ? s_max[lane] : 0u);
    const float m = __uint_as_float(mbits);
    const bool plain = m >= kLow && m <= kHigh;
    const float r = __fdiv_rn(127.0f, m);
    for (int g0 = 0; g0 < n_groups; g0 += T) {
        const int g = g0 + threadIdx.x;
        if constexpr (!kKeep) form(g, y);
        if (g < n_groups) {
            int8_t* dst = q + base + static_cast<int64_t>(g) * kVec;
            if (plain) {
                float far = 0.0f;
                *reinterpret_cast<uint2*>(dst) = quantize8(y, r, far);
                if (far > kNear)
                    decide8(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7], m, r, dst);
            } else {
                rare8(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7], mbits, dst);
            }
        }
        __syncwarp();
    }
    if (threadIdx.x == 0)
        scale[blockIdx.x] = mbits >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                                 : __fdiv_rn(m, 127.0f);
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

cudaError_t launch_gated_norm_i8(const GatedNormI8Args& a, cudaStream_t stream) {
    if (a.M == 0) return cudaSuccess;
    const int groups = a.Hv * (kDv / kVec);
    const int threads = std::min(1024, (groups + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const auto kernel = groups <= 1024 ? gated_norm_i8_kernel<true> : gated_norm_i8_kernel<false>;
    return cudaLaunchKernelEx(&cfg, kernel, a.o, a.z, a.norm_w, a.eps, a.q, a.scale, groups);
}

}  // namespace gdn
