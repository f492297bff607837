// gdn_linear_i8.cu -- y[M][N] = (x[M][K] . w[N][K]^T) * x_scale[m] * w_scale[n]
// on the sm_100a tensor cores: signed 8-bit operands, 32-bit integer sums,
// fp32 or bf16 out.
//
// The sums are integers and exact (K is at most 131056, so that K products of
// two bytes fit 32 bits): the tiling, the split of K and the order of its
// parts never show in a result. An element is converted to fp32 once and
// multiplied by the two scales in fp32.
//
// Three forms (plan_i8 in gdn_linear_i8_plan.h chooses by a model of their time):
//
//   vec    up to four tokens, and small products: dp4a on plain loads, no
//          barrier; bound by the weights' way from HBM (1 x 8192 x 8192 in
//          11.9 us, 5.7 TB/s) or by latency (1 x 64 x 2048 in 1.0 us);
//   split  tiles of 128 channels x 16 .. 128 tokens, one a CTA, K divided over
//          the CTAs of a cluster where there are few tiles: the weights are
//          the MMA's A operand, so that its width follows the tokens, and a
//          TMEM lane is an output channel. Bound by the chain setup - first
//          copy - MMAs - stores of a CTA (64 x 4096 x 2048 in 5.0 us, of which
//          the stores' and barriers' ends are 1.9 and a k-step of 256 bytes
//          0.29; the bytes' floor is 1.5);
//   pair   256 tokens x 128 or 256 channels over two SMs (cta_group::2),
//          persistent, a tile stored while the next one is formed: the tokens
//          are the A operand, so that a lane holds a token's neighbouring
//          channels and stores whole sectors. Bound by the tensor pipe at the
//          clock that the power limit leaves (8192^3 bf16 out, one cold call:
//          517 k cycles, 459 k of them MMA work, in 332 us, so 1.56 GHz and
//          3.3 POP/s), with short K by the stores beside it (16384 x 8192 x
//          2048: 174 to 181 us bf16, 213 to 256 us fp32 out, by that clock).
//
// What the loops cost decides the short kernels. An MMA of K = 32 bytes takes
// N / 2 cycles (at least 45), but a loop of one thread chosen by its lane
// number spent 411 cycles on issuing two tile loads and 446 on four MMAs; so
// whole warps run the loops, issue under elect_one(), ask for the next
// barrier before they issue (333), and a stage holds 256 bytes of K (257 a
// 128 bytes).
//
// Every mbarrier wait gives up after 2 s, ORs an error bit into the caller's
// status word (if given), lets copies in flight land and frees TMEM.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_linear_i8_plan.h"
#include "gdn_tc.cuh"
#include "gdn_tmap.h"

namespace gdn {

namespace {

constexpr int kAtom = 128;                   // bytes of K in a swizzled row
constexpr int kRows = kI8TileChannels;       // output channels of a split tile
constexpr int kThreads = 192;                // producer, MMA and four epilogue warps
constexpr int kMaxSplits = kI8MaxSplits;     // CTAs of a cluster

// ---- epilogue: integer sums to scaled fp32 or bf16 --------------------------
__device__ __forceinline__ float scaled(int acc, float sx, float sw) {
    // (acc * sx) first: the product of two small scales could lose bits below
    // the least normal number
    return __fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    __nv_bfloat162 b[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(b);
}

// 16 or 32 bytes at once (32: a whole sector), past L1: nothing here reads it
// again.
__device__ __forceinline__ void store16b(void* p, const uint32_t* u) {
    asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
}
__device__ __forceinline__ void store32b(void* p, const uint32_t* u) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]),
                   "r"(u[6]), "r"(u[7]) : "memory");
}
// The first `n` of a token's 32 channels, `align` (16 or 32) bytes at once: n
// is a whole number of such pieces.
template <typename YT>
__device__ __forceinline__ void store32(YT* p, const float (&v)[32], int n, int align) {
    constexpr int kWords = 32 * sizeof(YT) / 4, kPer = 4 / sizeof(YT);   // channels a word
    uint32_t u[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
        if constexpr (sizeof(YT) == 4) {
            u[j] = __float_as_uint(v[j]);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    if (align == 32) {
#pragma unroll
        for (int j = 0; j < kWords; j += 8)
            if (j * kPer < n) store32b(p + j * kPer, u + j);
    } else {
#pragma unroll
        for (int j = 0; j < kWords; j += 4)
            if (j * kPer < n) store16b(p + j * kPer, u + j);
    }
}
// v[j] of lane i becomes v[i] of lane j: at each step the lanes that differ in
// one bit swap the halves of their values that differ in it.
__device__ __forceinline__ void transpose32(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if ((j & o) == 0) {
                const float got = __shfl_xor_sync(kFull, up ? v[j] : v[j | o], o);
                if (up) v[j] = got; else v[j | o] = got;
            }
        }
    }
}

__device__ __forceinline__ void store2(float* p, float a, float b) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
// v[j] of each lane is token j's value of the warp's channel `lane`; y points
// at token 0's first one, `channels` and `left` tokens of them exist. `even`
// (N and y allow two channels at once): neighbouring lanes trade, so that a
// store covers two tokens with half as many stores (6000 x 1998 x 64 bf16 in
// 17.3 us against 21.4).
template <int kTokens, typename YT>
__device__ __forceinline__ void store_columns(YT* y, const float (&v)[kTokens], int64_t N,
                                              int channels, int left, int lane, bool even) {
    if (even) {
        const bool odd = lane & 1;
        YT* dst = y + (odd ? N : 0) + (lane & ~1);
        const bool have = lane < channels;
#pragma unroll
        for (int j = 0; j < kTokens; j += 2, dst += 2 * N) {
            const float got = __shfl_xor_sync(kFull, odd ? v[j] : v[j + 1], 1);
            if (have && j + (odd ? 1 : 0) < left)
                store2(dst, odd ? got : v[j], odd ? v[j + 1] : got);
        }
    } else if (lane < channels) {
        YT* dst = y + lane;
#pragma unroll
        for (int j = 0; j < kTokens; ++j, dst += N)
            if (j < left) store1(dst, v[j]);
    }
}

// A wait that ran out: reported, and seen by the CTA's other warps.
__device__ __forceinline__ void give_up(uint32_t* status, uint32_t bit, int* failed) {
    if ((threadIdx.x & 31) == 0) {
        if (status) atomicOr(status, bit);
        atomicExch(failed, 1);
    }
    __syncwarp();
}

// ---- split form --------------------------------------------------------------
// Sizes for MC tokens a tile: as many stages of 256 bytes of K as fit 192 KB.
template <int MC>
struct SplitSmem {
    static constexpr int kAtoms = 2;                          // of K a stage
    static constexpr uint32_t kW = kRows * kAtom;             // one atom of each operand
    static constexpr uint32_t kX = MC * kAtom;
    static constexpr uint32_t kStage = kAtoms * (kW + kX);
    static constexpr int kStages = 196608 / kStage;
    static constexpr uint32_t kRing = kStage * kStages;
    static constexpr uint32_t kPart = MC * kRows * 4;         // the parked partial tile
    static constexpr size_t kDynamic = (kRing > kPart ? kRing : kPart) + 1024;
    static constexpr uint32_t kCols = MC < 32 ? 32 : MC;      // TMEM columns
};

template <int MC, typename YT>
__global__ void __launch_bounds__(kThreads, 1)
linear_i8_split_kernel(const __grid_constant__ CUtensorMap tmap_x,
                       const __grid_constant__ CUtensorMap tmap_w,
                       const float* x_scale, const float* w_scale,
                       YT* __restrict__ y, int M, int N, int K, int splits,
                       uint32_t* __restrict__ status) {
    using L = SplitSmem<MC>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kStages];
    __shared__ __align__(8) uint64_t empty[kStages];
    __shared__ __align__(8) uint64_t acc_full;
    __shared__ __align__(16) float sx_s[4][MC];        // the tokens' scales, for each epilogue warp
    __shared__ __align__(16) float sw_s[kRows];        // the channels', for the cluster's sums
    __shared__ uint32_t tmem_slot;
    __shared__ int issued, consumed;
    __shared__ int failed;

    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    int* part = reinterpret_cast<int*>(smem_raw + (base - raw));   // [MC][128], after the MMAs

    const int warp = tc::warp_index();
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % splits;
    const int n_tiles = (N + kRows - 1) / kRows;
    const int tile = static_cast<int>(blockIdx.x) / splits;
    const int n0 = (tile % n_tiles) * kRows;
    const int m0 = (tile / n_tiles) * MC;
    constexpr int kBK = L::kAtoms * kAtom;
    const int n_kt = (K + kBK - 1) / kBK;
    const int kb = static_cast<int>(static_cast<int64_t>(rank) * n_kt / splits);
    const int ke = static_cast<int>(static_cast<int64_t>(rank + 1) * n_kt / splits);

    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&tmap_x);
        tc::prefetch_tmap(&tmap_w);
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(tc::smem_u32(&full[s]), 1);
            tc::mbar_init(tc::smem_u32(&empty[s]), 1);
        }
        tc::mbar_init(tc::smem_u32(&acc_full), 1);
        tc::fence_mbar_init();
        issued = 0;
        consumed = 0;
        failed = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc(tc::smem_u32(&tmem_slot), L::kCols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    tc::grid_dep_launch();
    int done = 0;                                      // k-steps issued, or consumed

    if (warp == 0) {
        if (tc::elect_one()) {
            // the first weight boxes head for L2 while the previous kernel ends
            tc::tma_prefetch_l2_2d(&tmap_w, kb * kBK, n0);
            if (kb * kBK + kAtom < K) tc::tma_prefetch_l2_2d(&tmap_w, kb * kBK + kAtom, n0);
        }
        tc::grid_dep_wait();
        int s = 0;
        uint32_t ph = 1;                               // the ring starts empty
        bool ready = true;
        for (int kt = kb; kt < ke; ++kt) {
            if (!__all_sync(kFull, ready) && !tc::mbar_wait_warp(tc::smem_u32(&empty[s]), ph)) {
                give_up(status, tc::kTimeoutProducer, &failed);
                break;
            }
            const uint32_t fb = tc::smem_u32(&full[s]);
            const uint32_t a = base + s * L::kStage;
            if (++s == kStages) { s = 0; ph ^= 1; }
            ready = tc::mbar_test_wait(tc::smem_u32(&empty[s]), ph);   // answered by the next pass
            // (past the end of K nothing is loaded, and no MMA is issued)
            const int left = K - kt * kBK;
            if (tc::elect_one()) {
                tc::mbar_arrive_expect_tx(fb, left > kAtom ? L::kStage : L::kW + L::kX);
#pragma unroll
                for (int i = 0; i < L::kAtoms; ++i) {
                    if (i * kAtom >= left) continue;
                    tc::tma_load_2d(a + i * L::kW, &tmap_w, fb, kt * kBK + i * kAtom, n0);
                    tc::tma_load_2d(a + L::kAtoms * L::kW + i * L::kX, &tmap_x, fb,
                                    kt * kBK + i * kAtom, m0);
                }
            }
            ++done;
        }
        if (lane == 0) issued = done;
    } else if (warp == 1) {
        tc::grid_dep_wait();
        const uint32_t idesc = tc::idesc_s8_s32(kRows, MC);
        int s = 0;
        uint32_t ph = 0;
        bool ready = false;
        for (int kt = kb; kt < ke; ++kt) {
            if (!__all_sync(kFull, ready) && !tc::mbar_wait_warp(tc::smem_u32(&full[s]), ph)) {
                give_up(status, tc::kTimeoutMma, &failed);
                break;
            }
            tc::tc_fence_after();
            const uint64_t a = tc::desc_k_sw128(base + s * L::kStage);
            const uint64_t b = tc::desc_k_sw128(base + s * L::kStage + L::kAtoms * L::kW);
            const uint32_t eb = tc::smem_u32(&empty[s]);
            if (++s == kStages) { s = 0; ph ^= 1; }
            ready = tc::mbar_test_wait(tc::smem_u32(&full[s]), ph);
            const int left = K - kt * kBK;
            if (tc::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk) {    // 32 bytes on: addresses count 16s
                    if (kk * 32 >= left) continue;
                    const int i = kk / 4, o = 2 * (kk % 4);
                    tc::mma_i8(tmem, a + (i * L::kW >> 4) + o, b + (i * L::kX >> 4) + o, idesc,
                               (kt > kb || kk > 0) ? 1u : 0u);
                }
                tc::mma_commit(eb);
                if (kt == ke - 1) tc::mma_commit(tc::smem_u32(&acc_full));
            }
            ++done;
        }
        if (lane == 0) consumed = done;
    } else if (warp >= 2) {
        tc::grid_dep_wait();
        const int quarter = warp & 3;                  // TMEM lanes 32 q .. 32 q + 31
        const int c = quarter * 32 + lane;             // this thread's channel of the tile
        const int tokens = min(MC, M - m0);
        const int n = n0 + c;
        // the scales come in while the MMAs run
        const float sw = n < N ? w_scale[n] : 0.0f;
        for (int j = lane; j < MC; j += 32)
            sx_s[warp - 2][j] = j < tokens ? x_scale[m0 + j] : 0.0f;
        if (splits > 1) sw_s[c] = sw;
        __syncwarp();
        if (!tc::mbar_wait_warp(tc::smem_u32(&acc_full), 0)) {
            give_up(status, tc::kTimeoutEpilogue, &failed);
        } else {
            tc::tc_fence_after();
            const uint32_t src = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            constexpr int kLd = MC < 32 ? 16 : 32;
            // (fp32 stores of single tokens are 128 bytes already: pairs took
            // 2% longer, and bf16 pairs 2% less; y is aligned to 16 bytes)
            const bool even = sizeof(YT) == 2 && (N & 1) == 0;
            // (rolled: unrolled, 128 tokens took 6100 cycles against 2000,
            // since each CTA waits for the code of every pass)
#pragma unroll 1
            for (int c0 = 0; c0 < tokens; c0 += kLd) {
                uint32_t r[kLd];
                if constexpr (kLd == 32) tc::tmem_ld_32x32b_x32(src + c0, r);
                else tc::tmem_ld_32x32b_x16(src + c0, r);
                tc::tmem_ld_wait();
                if (splits > 1) {
#pragma unroll
                    for (int j = 0; j < kLd; ++j)
                        part[(c0 + j) * kRows + c] = static_cast<int>(r[j]);
                } else {
                    float v[kLd];
#pragma unroll
                    for (int j = 0; j < kLd; j += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&sx_s[warp - 2][c0 + j]);
                        v[j] = scaled(static_cast<int>(r[j]), f.x, sw);
                        v[j + 1] = scaled(static_cast<int>(r[j + 1]), f.y, sw);
                        v[j + 2] = scaled(static_cast<int>(r[j + 2]), f.z, sw);
                        v[j + 3] = scaled(static_cast<int>(r[j + 3]), f.w, sw);
                    }
                    store_columns(y + static_cast<int64_t>(m0 + c0) * N + n - lane, v, N,
                                  N - (n - lane), tokens - c0, lane, even);
                    __syncwarp();
                }
            }
        }
    }

    __syncthreads();
    __syncwarp();
    if (splits > 1) {
        // every CTA adds its share of the tokens over the cluster's partials
        tc::cluster_sync();
        const int tokens = min(MC, M - m0);
        const uint32_t peer0 = tc::map_shared_rank(base, 0);
        const bool wide = (N & 3) == 0;
        const int n = n0 + 4 * lane;          // channels 4 lane .. 4 lane + 3 of the tile
        const float4 sw = *reinterpret_cast<const float4*>(&sw_s[4 * lane]);
        // (short code: each of these CTAs runs it a few times only, and what
        // it costs first is its instructions' way from memory)
#pragma unroll 1
        for (int m = rank + splits * warp; m < tokens; m += splits * (kThreads / 32)) {
            const float sx = sx_s[0][m];
            const uint32_t off = static_cast<uint32_t>((m * kRows + 4 * lane) * 4);
            int4 t = tc::ld_cluster_i4(peer0 + off);
            int4 v[kMaxSplits - 1];
#pragma unroll
            for (int p = 1; p < kMaxSplits; ++p)
                v[p - 1] = p < splits ? tc::ld_cluster_i4(tc::map_shared_rank(base + off, p))
                                      : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int p = 0; p < kMaxSplits - 1; ++p) {
                t.x += v[p].x; t.y += v[p].y; t.z += v[p].z; t.w += v[p].w;
            }
            const float o[4] = {scaled(t.x, sx, sw.x), scaled(t.y, sx, sw.y),
                                scaled(t.z, sx, sw.z), scaled(t.w, sx, sw.w)};
            YT* dst = y + static_cast<int64_t>(m0 + m) * N + n;
            if (wide) {
                if (n < N) store4(dst, o);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < N) store1(dst + j, o[j]);
            }
        }
        // no CTA leaves while a peer still reads its partial tile
        __syncwarp();
        tc::cluster_sync();
    }
    if (threadIdx.x == 0 && failed) {
        for (int g = consumed; g < issued; ++g)
            tc::mbar_wait(tc::smem_u32(&full[g % kStages]), static_cast<uint32_t>(g / kStages) & 1u);
    }
    tc::tc_fence_before();
    __syncthreads();
    __syncwarp();
    tc::tc_fence_after();
    if (warp == 1) tc::tmem_dealloc(tmem, L::kCols);
}

// ---- pair form ------------------------------------------------------------------
// A cluster of two CTAs owns a tile of 256 tokens x TN channels; the leader
// (rank 0) issues M = 256 MMAs. Each CTA stages its 128 rows of x and TN / 2
// of w per k-step and holds its 128 tokens of the accumulator, two sets of TN
// columns. Eight epilogue warps, a quarter of the lanes and half of the
// channels each (four: 235 against 231 us for 16384 x 8192 x 2048 fp32). They
// hand a set back with a plain arrive: a release at cluster scope first waits
// for the warp's stores (219 against 215 us).
//   full[s]    leader: one arrival (the leader's expect-tx of both CTAs'
//              bytes); both CTAs' loads complete on it
//   empty[s]   both: the leader's commit of the stage
//   acc_full   both: the leader's commit of the tile
//   acc_empty  leader: the eight epilogue warps of both CTAs
constexpr int kPairThreads = 64 + 8 * 32;             // two epilogue warps a TMEM lane quarter
template <int TN>
struct PairSmem {
    static constexpr int kAtoms = TN == 256 ? 1 : 2;     // of K a stage
    static constexpr uint32_t kX = 128 * kAtom;          // a CTA's half of the tokens, one atom
    static constexpr uint32_t kW = TN / 2 * kAtom;       // and of the channels
    static constexpr uint32_t kStage = kAtoms * (kX + kW);
    static constexpr int kStages = 196608 / kStage;
    static constexpr uint32_t kRing = kStage * kStages;
    static constexpr size_t kDynamic = kRing + 1024;
};

template <int TN, typename YT>
__global__ void __launch_bounds__(kPairThreads, 1)
linear_i8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ CUtensorMap tmap_w,
                      const float* x_scale, const float* w_scale,
                      YT* __restrict__ y, int align, int M, int N, int K,
                      uint32_t* __restrict__ status) {
    using L = PairSmem<TN>;
    constexpr int kPairStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kPairStages];
    __shared__ __align__(8) uint64_t empty[kPairStages];
    __shared__ __align__(8) uint64_t acc_full[2];
    __shared__ __align__(8) uint64_t acc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float sw_s[8][TN / 2];    // the scales of a warp's channels
    __shared__ int issued, consumed;
    __shared__ int failed;

    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const int warp = tc::warp_index();
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(tc::cluster_ctarank());   // 0: leader
    const int pair = static_cast<int>(blockIdx.x >> 1);
    const int n_pairs = static_cast<int>(gridDim.x >> 1);
    constexpr int kBK = L::kAtoms * kAtom;
    const int n_kt = (K + kBK - 1) / kBK;
    const int tiles_n = (N + TN - 1) / TN;
    const int n_tiles = tiles_n * ((M + 255) / 256);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            tc::mbar_init(tc::smem_u32(&full[s]), 1);
            tc::mbar_init(tc::smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(tc::smem_u32(&acc_full[a]), 1);
            tc::mbar_init(tc::smem_u32(&acc_empty[a]), 16);
        }
        tc::fence_mbar_init();
        issued = 0;
        consumed = 0;
        failed = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tc::smem_u32(&tmem_slot), 2 * TN);
        tc::tmem_relinquish_pair();
    }
    // both CTAs' barriers exist before either signals the other's
    tc::tc_fence_before();
    __syncthreads();
    __syncwarp();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    volatile int* vfailed = &failed;
    tc::grid_dep_launch();
    int done = 0;                                      // k-steps issued, or consumed

    if (warp == 0) {
        if (tc::elect_one()) {
            tc::prefetch_tmap(&tmap_x);
            tc::prefetch_tmap(&tmap_w);
        }
        tc::grid_dep_wait();
        const uint32_t full0 = tc::map_shared_rank(tc::smem_u32(&full[0]), 0);   // the leader's
        int s = 0;
        uint32_t ph = 1;
        bool ready = true;
        for (int tile = pair; tile < n_tiles && !__any_sync(kFull, *vfailed); tile += n_pairs) {
            const int m0 = (tile / tiles_n) * 256 + rank * 128;
            const int n0 = (tile % tiles_n) * TN + rank * (TN / 2);
            for (int kt = 0; kt < n_kt; ++kt) {
                if (!__all_sync(kFull, ready) && !tc::mbar_wait_warp(tc::smem_u32(&empty[s]), ph)) {
                    give_up(status, tc::kTimeoutProducer, &failed);
                    break;
                }
                const uint32_t a = base + s * L::kStage;
                const uint32_t fb = full0 + 8 * s;
                const uint32_t own = tc::smem_u32(&full[s]);
                if (++s == kPairStages) { s = 0; ph ^= 1; }
                ready = tc::mbar_test_wait(tc::smem_u32(&empty[s]), ph);   // for the next pass
                const int left = K - kt * kBK;
                if (tc::elect_one()) {
                    if (rank == 0)
                        tc::mbar_arrive_expect_tx(own, left > (L::kAtoms - 1) * kAtom
                                                           ? 2 * L::kStage : 2 * (L::kX + L::kW));
#pragma unroll
                    for (int i = 0; i < L::kAtoms; ++i) {
                        if (i * kAtom >= left) continue;
                        const int k0 = kt * kBK + i * kAtom;
                        tc::tma_load_2d_pair(a + i * L::kX, &tmap_x, fb, k0, m0);
                        tc::tma_load_2d_pair(a + L::kAtoms * L::kX + i * L::kW, &tmap_w, fb, k0, n0);
                    }
                }
                ++done;
            }
        }
        if (lane == 0) issued = done;
    } else if (warp == 1 && rank == 0) {
        tc::grid_dep_wait();
        const uint32_t idesc = tc::idesc_s8_s32(256, TN);
        int s = 0;
        uint32_t ph = 0;
        bool ready = false;
        bool ok = true;
        int li = 0;
        for (int tile = pair; ok && tile < n_tiles; tile += n_pairs, ++li) {
            const int acc = li & 1;
            const uint32_t d = tmem + static_cast<uint32_t>(acc) * TN;
            if (!tc::mbar_wait_warp(tc::smem_u32(&acc_empty[acc]), ((li >> 1) & 1) ^ 1)) {
                give_up(status, tc::kTimeoutMma, &failed);
                break;
            }
            tc::tc_fence_after();
            for (int kt = 0; kt < n_kt; ++kt) {
                if (!__all_sync(kFull, ready) && !tc::mbar_wait_warp(tc::smem_u32(&full[s]), ph)) {
                    give_up(status, tc::kTimeoutMma, &failed);
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
                const uint64_t a = tc::desc_k_sw128(base + s * L::kStage);
                const uint64_t b = tc::desc_k_sw128(base + s * L::kStage + L::kAtoms * L::kX);
                const uint32_t eb = tc::smem_u32(&empty[s]);
                if (++s == kPairStages) { s = 0; ph ^= 1; }
                ready = tc::mbar_test_wait(tc::smem_u32(&full[s]), ph);
                const int left = K - kt * kBK;
                if (tc::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk) {
                        if (kk * 32 >= left) continue;
                        const int i = kk / 4, o = 2 * (kk % 4);
                        tc::mma_i8_pair(d, a + (i * L::kX >> 4) + o, b + (i * L::kW >> 4) + o, idesc,
                                        (kt > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc::mma_commit_pair(eb, 0x3);
                    if (kt == n_kt - 1) tc::mma_commit_pair(tc::smem_u32(&acc_full[acc]), 0x3);
                }
                ++done;
            }
        }
        if (lane == 0) consumed = done;
    } else if (warp >= 2) {
        tc::grid_dep_wait();
        const int quarter = warp & 3;                  // TMEM lanes 32 q .. 32 q + 31
        const int col0 = (warp - 2) / 4 * (TN / 2);    // and half of the tile's channels
        const uint32_t ae0 = tc::map_shared_rank(tc::smem_u32(&acc_empty[0]), 0);
        const uint32_t ae1 = tc::map_shared_rank(tc::smem_u32(&acc_empty[1]), 0);
        int li = 0;
        for (int tile = pair; tile < n_tiles; tile += n_pairs, ++li) {
            const int acc = li & 1;
            const int row = (tile / tiles_n) * 256 + rank * 128 + quarter * 32 + lane;   // token
            const int n0 = (tile % tiles_n) * TN + col0;
            const int channels = min(TN / 2, N - n0);  // 0 or less: nothing but the hand-over
            const float sx = row < M ? x_scale[row] : 0.0f;
            float* sws = sw_s[warp - 2];
#pragma unroll
            for (int j = 0; j < TN / 2; j += 32)
                sws[j + lane] = j + lane < channels ? w_scale[n0 + j + lane] : 0.0f;
            __syncwarp();
            const uint32_t src = tmem + static_cast<uint32_t>(acc) * TN + col0 +
                                 (static_cast<uint32_t>(quarter * 32) << 16);
            if (!tc::mbar_wait_warp(tc::smem_u32(&acc_full[acc]), (li >> 1) & 1)) {
                give_up(status, tc::kTimeoutEpilogue, &failed);
                break;
            }
            tc::tc_fence_after();
            if (channels <= 0 && lane == 0) tc::mbar_arrive_cluster_local(acc ? ae1 : ae0);
#pragma unroll 1
            for (int c0 = 0; c0 < channels; c0 += 32) {
                uint32_t r[32];
                tc::tmem_ld_32x32b_x32(src + c0, r);
                tc::tmem_ld_wait();
                if (c0 + 32 >= channels) {        // every read of this set is done: hand it back
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cluster_local(acc ? ae1 : ae0);
                }
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(sws + c0 + j);
                    v[j] = scaled(static_cast<int>(r[j]), sx, f.x);
                    v[j + 1] = scaled(static_cast<int>(r[j + 1]), sx, f.y);
                    v[j + 2] = scaled(static_cast<int>(r[j + 2]), sx, f.z);
                    v[j + 3] = scaled(static_cast<int>(r[j + 3]), sx, f.w);
                }
                if (align >= 16) {
                    if (row < M)
                        store32(y + static_cast<int64_t>(row) * N + n0 + c0, v, channels - c0, align);
                } else {
                    // rows that are not aligned: one or two tokens' 32 channels a store
                    transpose32(v, lane);
                    store_columns(y + static_cast<int64_t>(row - lane) * N + n0 + c0, v, N,
                                  channels - c0, M - (row - lane), lane, (N & 1) == 0);
                }
                __syncwarp();
            }
            __syncwarp();
        }
    }

    // Both CTAs meet here; then the leader lets copies still addressed to its
    // barriers land (after a timeout only), and both meet again before TMEM
    // and shared memory are released.
    if (warp == 1 && rank != 0) tc::grid_dep_wait();
    tc::tc_fence_before();
    __syncthreads();
    __syncwarp();
    tc::cluster_sync();
    if (threadIdx.x == 0 && rank == 0 && failed) {
        for (int g = consumed; g < issued; ++g)
            tc::mbar_wait(tc::smem_u32(&full[g % kPairStages]),
                          static_cast<uint32_t>(g / kPairStages) & 1u);
    }
    __syncthreads();
    __syncwarp();
    tc::cluster_sync();
    tc::tc_fence_after();
    if (warp == 1) tc::tmem_dealloc_pair(tmem, 2 * TN);
}

// ---- few tokens --------------------------------------------------------------------
// The weights are read once and everything else is small: a warp reads R rows
// of w in 16-byte pieces, multiplies them with MT tokens' bytes four at a time
// and adds over its lanes. Nothing is shared between warps, so there is no
// barrier, and the weights of every warp are on their way at once.
constexpr int kVecThreads = 128;

__device__ __forceinline__ int4 ld_stream_i4(const int8_t* p) {
    int4 v;
    asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <int MT, int R, int W, typename YT>
__global__ void __launch_bounds__(kVecThreads)
linear_i8_vec_kernel(const int8_t* x, const float* x_scale, const int8_t* w,
                     const float* w_scale, YT* __restrict__ y, int M, int N, int K, int n_blocks) {
    constexpr int kWarps = kVecThreads / 32;
    constexpr int U = 2;                               // pieces of a row in flight
    constexpr int kSpan = 512 * W;                     // bytes that W warps read at once
    static_assert(MT * R <= 32, "a lane for each sum");
    __shared__ int part[W > 1 ? kWarps : 1][MT * R];
    const int lane = threadIdx.x & 31;
    const int warp = tc::warp_index();
    const int n0 = (static_cast<int>(blockIdx.x) % n_blocks * (kWarps / W) + warp / W) * R;
    const int m0 = static_cast<int>(blockIdx.x) / n_blocks * MT;
    const int at = warp % W * 32 + lane;               // this thread's place in a row
    tc::grid_dep_launch();
    const int8_t* wr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wr[r] = w + static_cast<int64_t>(min(n0 + r, N - 1)) * K;
    // the weights head for L2 while the previous kernel ends
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (at * 128 < K) asm volatile("prefetch.global.L2 [%0];" ::"l"(wr[r] + at * 128));
    tc::grid_dep_wait();
    // lane m R + r will keep the sum of token m0 + m and channel n0 + r; their
    // scales are on their way beside the operands (behind the sums: 2.7 against
    // 2.5 us for 256 x 64 x 2048, 4.6 against 4.2 for 8 x 2048 x 4096)
    const int my_m = m0 + lane / R, my_n = n0 + lane % R;
    const bool have = lane < MT * R && my_m < M && my_n < N;
    const float sx = have ? x_scale[my_m] : 0.0f, sw = have ? w_scale[my_n] : 0.0f;
    const int8_t* xr[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xr[m] = x + static_cast<int64_t>(min(m0 + m, M - 1)) * K;
    int acc[MT][R] = {};
    // `pieces` pieces of 16 bytes a thread, all loads first
    auto step = [&](int k, auto pieces) {
        constexpr int P = decltype(pieces)::value;
        int4 wv[P][R], xv[P][MT];
#pragma unroll
        for (int u = 0; u < P; ++u) {
#pragma unroll
            for (int r = 0; r < R; ++r) wv[u][r] = ld_stream_i4(wr[r] + k + kSpan * u);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                xv[u][m] = *reinterpret_cast<const int4*>(xr[m] + k + kSpan * u);
        }
#pragma unroll
        for (int u = 0; u < P; ++u) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[m][r] = __dp4a(wv[u][r].x, xv[u][m].x, acc[m][r]);
                    acc[m][r] = __dp4a(wv[u][r].y, xv[u][m].y, acc[m][r]);
                    acc[m][r] = __dp4a(wv[u][r].z, xv[u][m].z, acc[m][r]);
                    acc[m][r] = __dp4a(wv[u][r].w, xv[u][m].w, acc[m][r]);
                }
            }
        }
    };
    int k = at * 16;
    for (; k + kSpan * (U - 1) < K; k += kSpan * U) step(k, std::integral_constant<int, U>{});
    for (; k < K; k += kSpan) step(k, std::integral_constant<int, 1>{});
    int mine = 0;
#pragma unroll
    for (int i = 0; i < MT * R; ++i) {
        const int t = __reduce_add_sync(kFull, acc[i / R][i % R]);
        if (lane == i) mine = t;
    }
    if constexpr (W > 1) {
        if (lane < MT * R) part[warp][lane] = mine;
        __syncthreads();
        if (warp % W != 0) return;
        if (lane < MT * R) {
#pragma unroll
            for (int i = 1; i < W; ++i) mine += part[warp + i][lane];
        }
    }
    if (have) store1(y + static_cast<int64_t>(my_m) * N + my_n, scaled(mine, sx, sw));
}

// ---- host ------------------------------------------------------------------------
// Row-major [rows][K] bytes as a 2D tensor map with box [box_rows][128].
bool make_tmap_i8(CUtensorMap* map, const void* ptr, int64_t rows, int64_t K, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kAtom), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Raises the kernel's shared-memory limit (at every launch: it belongs to the
// context, which a program may replace).
cudaError_t allow_smem(const void* kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(bytes));
}

cudaLaunchConfig_t cluster_config(unsigned grid, int threads, int cluster, size_t smem,
                                  cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

template <int MC, typename YT>
cudaError_t launch_split(const LinearI8Args& a, int splits, cudaStream_t stream) {
    const auto kernel = linear_i8_split_kernel<MC, YT>;
    cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), SplitSmem<MC>::kDynamic);
    if (err != cudaSuccess) return err;
    CUtensorMap tx, tw;
    if (!make_tmap_i8(&tx, a.x, a.M, a.K, MC) || !make_tmap_i8(&tw, a.w, a.N, a.K, kRows))
        return cudaErrorInvalidValue;
    const int64_t ctas = ((a.N + kRows - 1) / kRows) * ((a.M + MC - 1) / MC) * splits;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(static_cast<unsigned>(ctas), kThreads, splits,
                                                  SplitSmem<MC>::kDynamic, stream, attr);
    return cudaLaunchKernelEx(&cfg, kernel, tx, tw, a.x_scale, a.w_scale, static_cast<YT*>(a.y),
                              static_cast<int>(a.M), static_cast<int>(a.N),
                              static_cast<int>(a.K), splits, a.status);
}

template <int TN, typename YT>
cudaError_t launch_pair(const LinearI8Args& a, cudaStream_t stream) {
    const auto kernel = linear_i8_pair_kernel<TN, YT>;
    cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), PairSmem<TN>::kDynamic);
    if (err != cudaSuccess) return err;
    CUtensorMap tx, tw;
    if (!make_tmap_i8(&tx, a.x, a.M, a.K, 128) || !make_tmap_i8(&tw, a.w, a.N, a.K, TN / 2))
        return cudaErrorInvalidValue;
    const int64_t tiles = ((a.N + TN - 1) / TN) * ((a.M + 255) / 256);
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int64_t pairs = std::min<int64_t>(tiles, device_sm_count() / 2);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(static_cast<unsigned>(2 * pairs), kPairThreads, 2,
                                                  PairSmem<TN>::kDynamic, stream, attr);
    const uint64_t rows = (a.N * sizeof(YT)) | reinterpret_cast<uintptr_t>(a.y);   // their alignment
    return cudaLaunchKernelEx(&cfg, kernel, tx, tw, a.x_scale, a.w_scale,
                              static_cast<YT*>(a.y),
                              rows % 32 == 0 ? 32 : rows % 16 == 0 ? 16 : 0, static_cast<int>(a.M),
                              static_cast<int>(a.N), static_cast<int>(a.K), a.status);
}

template <int MT, int R, int W, typename YT>
cudaError_t launch_vec_r(const LinearI8Args& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    const int64_t rows = kVecThreads / 32 / W * R;
    const int64_t n_blocks = (a.N + rows - 1) / rows, blocks = n_blocks * ((a.M + MT - 1) / MT);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kVecThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_i8_vec_kernel<MT, R, W, YT>, a.x, a.x_scale, a.w,
                              a.w_scale, static_cast<YT*>(a.y), static_cast<int>(a.M),
                              static_cast<int>(a.N), static_cast<int>(a.K),
                              static_cast<int>(n_blocks));
}

template <int MT, int R, typename YT>
cudaError_t launch_vec_w(const LinearI8Args& a, cudaStream_t stream) {
    switch (vec_warps(a.K)) {
        case 4: return launch_vec_r<MT, R, 4, YT>(a, stream);
        case 2: return launch_vec_r<MT, R, 2, YT>(a, stream);
        default: return launch_vec_r<MT, R, 1, YT>(a, stream);
    }
}

// R rows a warp: as many as keep its loads few without leaving it too few in
// flight (8 x 2048 x 4096: 4.2 with 4 against 4.6 with 2; 1 x 1000 x 10000: 3.4
// with 2, 4.6 with 4). Where another number is better: 8 x 4096 x 2048 takes 4.5
// with 2 and 4.1 with 4.
template <typename YT>
cudaError_t launch_vec(const LinearI8Args& a, cudaStream_t stream) {
    if (a.M <= 1) return launch_vec_w<1, 2, YT>(a, stream);
    if (a.M <= 2) return launch_vec_w<2, 2, YT>(a, stream);
    if (a.M <= 4) return launch_vec_w<4, 4, YT>(a, stream);
    if (vec_warps(a.K) == 4) return launch_vec_r<8, 4, 4, YT>(a, stream);
    if (vec_warps(a.K) == 2) return launch_vec_r<8, 2, 2, YT>(a, stream);
    return launch_vec_r<8, 2, 1, YT>(a, stream);
}

template <typename YT>
cudaError_t launch_typed(const LinearI8Args& a, cudaStream_t stream) {
    const PlanI8 p = plan_i8(a.M, a.N, a.K, device_sm_count());
    if (p.form == PlanI8::kVec) return launch_vec<YT>(a, stream);
    if (p.form == PlanI8::kPair)
        return p.tile == 256 ? launch_pair<256, YT>(a, stream) : launch_pair<128, YT>(a, stream);
    switch (p.tile) {
        case 16: return launch_split<16, YT>(a, p.splits, stream);
        case 32: return launch_split<32, YT>(a, p.splits, stream);
        case 64: return launch_split<64, YT>(a, p.splits, stream);
        default: return launch_split<128, YT>(a, p.splits, stream);
    }
}

}  // namespace

cudaError_t launch_linear_i8(const LinearI8Args& a, cudaStream_t stream) {
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    return a.y_bf16 ? launch_typed<__nv_bfloat16>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace gdn
