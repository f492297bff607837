// gdn_linear_i8.cu -- y[M][N] = (x[M][K] . w[N][K]^T) * x_scale[m] * w_scale[n]
// on the sm_100a tensor cores: signed 8-bit operands, 32-bit integer sums,
// fp32 or bf16 out.
//
// The sums are integers and exact (K is at most 131056, so that K products of
// two bytes fit 32 bits): the tiling, the split of K and the order of its
// parts never show in a result. An element is converted to fp32 once and
// multiplied by the two scales in fp32.
//
// The weights are the MMA's A operand (128 or 256 rows of D are output
// channels) and the tokens its B operand (the columns of D): a decode-sized
// call then has an MMA as narrow as its few tokens, and since a TMEM lane is
// an output channel, a warp's store of one token's 32 channels is contiguous.
//
//   split form  128 channels x MC tokens a tile (MC = 16 .. 256), K divided
//               over the S CTAs of a cluster, whose partial tiles are added
//               through distributed shared memory;
//   pair form   256 x 256 tiles over pairs of SMs (cta_group::2), persistent,
//               two accumulator sets so that a tile drains under the next.
//
// Every mbarrier wait gives up after 2 s, ORs an error bit into the caller's
// status word (if given), lets copies in flight land and frees TMEM.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tmap.h"

namespace gdn {

namespace {

constexpr int kBK = 128;                     // bytes of K a stage: one swizzle row
constexpr int kRows = 128;                   // output channels of a split tile
constexpr int kThreads = 192;                // producer, MMA and four epilogue warps
constexpr int kMaxSplits = 8;                // CTAs of a cluster

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

// ---- split form --------------------------------------------------------------
template <int MC>
struct SplitSmem {
    static constexpr uint32_t kW = kRows * kBK;
    static constexpr uint32_t kStage = kW + MC * kBK;
    static constexpr int kStages = (196608 / kStage) < 10 ? static_cast<int>(196608 / kStage) : 10;
    static constexpr uint32_t kRing = kStage * kStages;
    static constexpr uint32_t kPart = MC * kRows * 4;         // the parked partial tile
    static constexpr size_t kDynamic = (kRing > kPart ? kRing : kPart) + 1024;
    static constexpr uint32_t kCols = MC < 32 ? 32 : MC;      // TMEM columns
};

template <int MC, typename YT>
__global__ void __launch_bounds__(kThreads, 1)
linear_i8_split_kernel(const __grid_constant__ CUtensorMap tmap_x,
                       const __grid_constant__ CUtensorMap tmap_w,
                       const float* __restrict__ x_scale, const float* __restrict__ w_scale,
                       YT* __restrict__ y, int M, int N, int K, int splits,
                       uint32_t* __restrict__ status) {
    using L = SplitSmem<MC>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kStages];
    __shared__ __align__(8) uint64_t empty[kStages];
    __shared__ __align__(8) uint64_t acc_full;
    __shared__ uint32_t tmem_slot;
    __shared__ int issued, consumed;
    __shared__ int failed;

    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    int* part = reinterpret_cast<int*>(smem_raw + (base - raw));   // [MC][128], after the MMAs

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % splits;
    const int n_tiles = (N + kRows - 1) / kRows;
    const int tile = static_cast<int>(blockIdx.x) / splits;
    const int n0 = (tile % n_tiles) * kRows;
    const int m0 = (tile / n_tiles) * MC;
    const int n_kt = (K + kBK - 1) / kBK;
    const int kb = static_cast<int>(static_cast<int64_t>(rank) * n_kt / splits);
    const int ke = static_cast<int>(static_cast<int64_t>(rank + 1) * n_kt / splits);

    if (threadIdx.x == 0) {
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

    if (warp == 0 && lane == 0) {
        tc::prefetch_tmap(&tmap_x);
        tc::prefetch_tmap(&tmap_w);
        // the first weight boxes head for L2 while the previous kernel ends
        for (int kt = kb; kt < ke && kt < kb + 2; ++kt) tc::tma_prefetch_l2_2d(&tmap_w, kt * kBK, n0);
        tc::grid_dep_wait();
        int s = 0;
        uint32_t ph = 1;                               // the ring starts empty
        for (int kt = kb; kt < ke; ++kt) {
            const uint32_t fb = tc::smem_u32(&full[s]);
            if (!tc::mbar_wait(tc::smem_u32(&empty[s]), ph)) {
                if (status) atomicOr(status, tc::kTimeoutProducer);
                atomicExch(&failed, 1);
                break;
            }
            const uint32_t a = base + s * L::kStage;
            tc::mbar_arrive_expect_tx(fb, L::kStage);
            tc::tma_load_2d(a, &tmap_w, fb, kt * kBK, n0);
            tc::tma_load_2d(a + L::kW, &tmap_x, fb, kt * kBK, m0);
            issued = kt - kb + 1;
            if (++s == kStages) { s = 0; ph ^= 1; }
        }
    } else if (warp == 1 && lane == 0) {
        tc::grid_dep_wait();
        const uint32_t idesc = tc::idesc_s8_s32(kRows, MC);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int kt = kb; kt < ke; ++kt) {
            if (!tc::mbar_wait(tc::smem_u32(&full[s]), ph)) {
                if (status) atomicOr(status, tc::kTimeoutMma);
                atomicExch(&failed, 1);
                ok = false;
                break;
            }
            consumed = kt - kb + 1;
            tc::tc_fence_after();
            const uint64_t a = tc::desc_k_sw128(base + s * L::kStage);
            const uint64_t b = tc::desc_k_sw128(base + s * L::kStage + L::kW);
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)      // 32 bytes on: the address field counts 16s
                tc::mma_i8(tmem, a + 2 * kk, b + 2 * kk, idesc, (kt > kb || kk > 0) ? 1u : 0u);
            tc::mma_commit(tc::smem_u32(&empty[s]));
            if (++s == kStages) { s = 0; ph ^= 1; }
        }
        if (ok) tc::mma_commit(tc::smem_u32(&acc_full));
    } else if (warp >= 2) {
        tc::grid_dep_wait();
        const int quarter = warp & 3;                  // TMEM lanes 32 q .. 32 q + 31
        const int c = quarter * 32 + lane;             // this thread's channel of the tile
        if (!tc::mbar_wait(tc::smem_u32(&acc_full), 0)) {
            if (status) atomicOr(status, tc::kTimeoutEpilogue);
            atomicExch(&failed, 1);
        } else {
            tc::tc_fence_after();
            const uint32_t src = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            const int tokens = min(MC, M - m0);
            const int n = n0 + c;
            const float sw = splits == 1 && n < N ? w_scale[n] : 0.0f;
            constexpr int kLd = MC < 32 ? 16 : 32;
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
                } else if (n < N) {
#pragma unroll
                    for (int j = 0; j < kLd; ++j)
                        if (c0 + j < tokens)
                            store1(y + static_cast<int64_t>(m0 + c0 + j) * N + n,
                                   scaled(static_cast<int>(r[j]), x_scale[m0 + c0 + j], sw));
                }
                __syncwarp();
            }
        }
    }

    if (warp < 2 && lane != 0) tc::grid_dep_wait();
    __syncthreads();
    __syncwarp();
    if (splits > 1) {
        // every CTA adds its share of the tokens over the cluster's partials
        tc::cluster_sync();
        const int tokens = min(MC, M - m0);
        uint32_t peer[kMaxSplits];
#pragma unroll
        for (int p = 0; p < kMaxSplits; ++p)
            peer[p] = p < splits ? tc::map_shared_rank(base, static_cast<uint32_t>(p)) : 0;
        const bool wide = (N & 3) == 0;
        // wide: channels 4 lane .. 4 lane + 3 of the tile
        float sw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + 4 * lane + j;
            sw[j] = n < N ? w_scale[n] : 0.0f;
        }
        const int n = n0 + 4 * lane;
#pragma unroll 1
        for (int m = rank + splits * warp; m < tokens; m += splits * (kThreads / 32)) {
            const uint32_t off = static_cast<uint32_t>((m * kRows + 4 * lane) * 4);
            int4 v[kMaxSplits];
#pragma unroll
            for (int p = 0; p < kMaxSplits; ++p)
                if (p < splits) v[p] = tc::ld_cluster_i4(peer[p] + off);
            int4 t = make_int4(0, 0, 0, 0);
#pragma unroll
            for (int p = 0; p < kMaxSplits; ++p) {
                if (p < splits) {
                    t.x += v[p].x; t.y += v[p].y; t.z += v[p].z; t.w += v[p].w;
                }
            }
            const float sx = x_scale[m0 + m];
            const float o[4] = {scaled(t.x, sx, sw[0]), scaled(t.y, sx, sw[1]),
                                scaled(t.z, sx, sw[2]), scaled(t.w, sx, sw[3])};
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
// A cluster of two CTAs owns a tile of 256 channels x 256 tokens; the leader
// (rank 0) issues M = 256 MMAs. Each CTA stages its 128 rows of w and of x per
// k-step and holds its 128 channels of the accumulator, two sets of 256
// columns.
//   full[s]    leader: one arrival (the leader's expect-tx of both CTAs'
//              bytes); both CTAs' loads complete on it
//   empty[s]   both: the leader's commit of the stage
//   acc_full   both: the leader's commit of the tile
//   acc_empty  leader: the four epilogue warps of both CTAs
constexpr int kPairStages = 6;
constexpr uint32_t kPairHalf = 128 * kBK;
constexpr uint32_t kPairStage = 2 * kPairHalf;
constexpr size_t kPairDynamic = static_cast<size_t>(kPairStage) * kPairStages + 1024;

template <typename YT>
__global__ void __launch_bounds__(kThreads, 1)
linear_i8_pair_kernel(const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ CUtensorMap tmap_w,
                      const float* __restrict__ x_scale, const float* __restrict__ w_scale,
                      YT* __restrict__ y, int M, int N, int K, uint32_t* __restrict__ status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kPairStages];
    __shared__ __align__(8) uint64_t empty[kPairStages];
    __shared__ __align__(8) uint64_t acc_full[2];
    __shared__ __align__(8) uint64_t acc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int issued, consumed;
    __shared__ int failed;

    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(tc::cluster_ctarank());   // 0: leader
    const int pair = static_cast<int>(blockIdx.x >> 1);
    const int n_pairs = static_cast<int>(gridDim.x >> 1);
    const int n_kt = (K + kBK - 1) / kBK;
    const int tiles_n = (N + 255) / 256;
    const int n_tiles = tiles_n * ((M + 255) / 256);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            tc::mbar_init(tc::smem_u32(&full[s]), 1);
            tc::mbar_init(tc::smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(tc::smem_u32(&acc_full[a]), 1);
            tc::mbar_init(tc::smem_u32(&acc_empty[a]), 8);
        }
        tc::fence_mbar_init();
        issued = 0;
        consumed = 0;
        failed = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tc::smem_u32(&tmem_slot), 512);
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

    if (warp == 0 && lane == 0) {
        tc::prefetch_tmap(&tmap_x);
        tc::prefetch_tmap(&tmap_w);
        tc::grid_dep_wait();
        int s = 0, g = 0;
        uint32_t ph = 1;
        for (int tile = pair; tile < n_tiles && !*vfailed; tile += n_pairs) {
            const int m0 = (tile / tiles_n) * 256 + rank * 128;
            const int n0 = (tile % tiles_n) * 256 + rank * 128;
            for (int kt = 0; kt < n_kt; ++kt) {
                if (!tc::mbar_wait(tc::smem_u32(&empty[s]), ph)) {
                    if (status) atomicOr(status, tc::kTimeoutProducer);
                    atomicExch(&failed, 1);
                    break;
                }
                const uint32_t a = base + s * kPairStage;
                const uint32_t fb = tc::map_shared_rank(tc::smem_u32(&full[s]), 0);
                if (rank == 0) tc::mbar_arrive_expect_tx(tc::smem_u32(&full[s]), 2 * kPairStage);
                tc::tma_load_2d_pair(a, &tmap_w, fb, kt * kBK, n0);
                tc::tma_load_2d_pair(a + kPairHalf, &tmap_x, fb, kt * kBK, m0);
                issued = ++g;
                if (++s == kPairStages) { s = 0; ph ^= 1; }
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        tc::grid_dep_wait();
        const uint32_t idesc = tc::idesc_s8_s32(256, 256);
        int s = 0, g = 0;
        uint32_t ph = 0;
        bool ok = true;
        int li = 0;
        for (int tile = pair; ok && tile < n_tiles; tile += n_pairs, ++li) {
            const int acc = li & 1;
            const uint32_t d = tmem + static_cast<uint32_t>(acc) * 256;
            if (!tc::mbar_wait(tc::smem_u32(&acc_empty[acc]), ((li >> 1) & 1) ^ 1)) {
                if (status) atomicOr(status, tc::kTimeoutMma);
                atomicExch(&failed, 1);
                break;
            }
            tc::tc_fence_after();
            for (int kt = 0; kt < n_kt; ++kt) {
                if (!tc::mbar_wait(tc::smem_u32(&full[s]), ph)) {
                    if (status) atomicOr(status, tc::kTimeoutMma);
                    atomicExch(&failed, 1);
                    ok = false;
                    break;
                }
                consumed = ++g;
                tc::tc_fence_after();
                const uint64_t a = tc::desc_k_sw128(base + s * kPairStage);
                const uint64_t b = tc::desc_k_sw128(base + s * kPairStage + kPairHalf);
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk)
                    tc::mma_i8_pair(d, a + 2 * kk, b + 2 * kk, idesc, (kt > 0 || kk > 0) ? 1u : 0u);
                tc::mma_commit_pair(tc::smem_u32(&empty[s]), 0x3);
                if (++s == kPairStages) { s = 0; ph ^= 1; }
            }
            if (ok) tc::mma_commit_pair(tc::smem_u32(&acc_full[acc]), 0x3);
        }
    } else if (warp >= 2) {
        tc::grid_dep_wait();
        const int quarter = warp & 3;
        const uint32_t ae0 = tc::map_shared_rank(tc::smem_u32(&acc_empty[0]), 0);
        const uint32_t ae1 = tc::map_shared_rank(tc::smem_u32(&acc_empty[1]), 0);
        int li = 0;
        for (int tile = pair; tile < n_tiles; tile += n_pairs, ++li) {
            const int acc = li & 1;
            if (!tc::mbar_wait(tc::smem_u32(&acc_full[acc]), (li >> 1) & 1)) {
                if (status) atomicOr(status, tc::kTimeoutEpilogue);
                atomicExch(&failed, 1);
                break;
            }
            tc::tc_fence_after();
            const int m0 = (tile / tiles_n) * 256;
            const int n = (tile % tiles_n) * 256 + rank * 128 + quarter * 32 + lane;
            const int tokens = min(256, M - m0);
            const float sw = n < N ? w_scale[n] : 0.0f;
            const uint32_t src = tmem + static_cast<uint32_t>(acc) * 256 +
                                 (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
            for (int c0 = 0; c0 < tokens; c0 += 32) {
                uint32_t r[32];
                tc::tmem_ld_32x32b_x32(src + c0, r);
                tc::tmem_ld_wait();
                if (n < N) {
                    YT* dst = y + static_cast<int64_t>(m0 + c0) * N + n;
#pragma unroll
                    for (int j = 0; j < 32; ++j, dst += N)
                        if (c0 + j < tokens)
                            store1(dst, scaled(static_cast<int>(r[j]), x_scale[m0 + c0 + j], sw));
                }
                __syncwarp();
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(acc ? ae1 : ae0);   // the leader's set is free
        }
    }

    // Both CTAs meet here; then the leader lets copies still addressed to its
    // barriers land (after a timeout only), and both meet again before TMEM
    // and shared memory are released.
    if (warp < 2 && (lane != 0 || (warp == 1 && rank != 0))) tc::grid_dep_wait();
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
    if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
}

// ---- host ------------------------------------------------------------------------
// Row-major [rows][K] bytes as a 2D tensor map with box [box_rows][128].
bool make_tmap_i8(CUtensorMap* map, const void* ptr, int64_t rows, int64_t K, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBK), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

constexpr int kDevs = 16;

// Raises the kernel's shared-memory limit once per device.
cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<bool> (&done)[kDevs]) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < kDevs && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(bytes));
    if (err == cudaSuccess && dev < kDevs) done[dev].store(true, std::memory_order_release);
    return err;
}

cudaLaunchConfig_t cluster_config(unsigned grid, int cluster, size_t smem, cudaStream_t stream,
                                  cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
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
    static std::atomic<bool> done[kDevs];
    const auto kernel = linear_i8_split_kernel<MC, YT>;
    cudaError_t err =
        allow_smem(reinterpret_cast<const void*>(kernel), SplitSmem<MC>::kDynamic, done);
    if (err != cudaSuccess) return err;
    CUtensorMap tx, tw;
    if (!make_tmap_i8(&tx, a.x, a.M, a.K, MC) || !make_tmap_i8(&tw, a.w, a.N, a.K, kRows))
        return cudaErrorInvalidValue;
    const int64_t ctas = ((a.N + kRows - 1) / kRows) * ((a.M + MC - 1) / MC) * splits;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(static_cast<unsigned>(ctas), splits,
                                                  SplitSmem<MC>::kDynamic, stream, attr);
    return cudaLaunchKernelEx(&cfg, kernel, tx, tw, a.x_scale, a.w_scale, static_cast<YT*>(a.y),
                              static_cast<int>(a.M), static_cast<int>(a.N),
                              static_cast<int>(a.K), splits, a.status);
}

template <typename YT>
cudaError_t launch_pair(const LinearI8Args& a, cudaStream_t stream) {
    static std::atomic<bool> done[kDevs];
    const auto kernel = linear_i8_pair_kernel<YT>;
    cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), kPairDynamic, done);
    if (err != cudaSuccess) return err;
    CUtensorMap tx, tw;
    if (!make_tmap_i8(&tx, a.x, a.M, a.K, 128) || !make_tmap_i8(&tw, a.w, a.N, a.K, 128))
        return cudaErrorInvalidValue;
    const int64_t tiles = ((a.N + 255) / 256) * ((a.M + 255) / 256);
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int64_t pairs = std::min<int64_t>(tiles, device_sm_count() / 2);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        cluster_config(static_cast<unsigned>(2 * pairs), 2, kPairDynamic, stream, attr);
    return cudaLaunchKernelEx(&cfg, kernel, tx, tw, a.x_scale, a.w_scale, static_cast<YT*>(a.y),
                              static_cast<int>(a.M), static_cast<int>(a.N),
                              static_cast<int>(a.K), a.status);
}

template <typename YT>
cudaError_t launch_typed(const LinearI8Args& a, cudaStream_t stream) {
    const int64_t sms = device_sm_count();
    const int64_t n_kt = (a.K + kBK - 1) / kBK;
    const int64_t pair_tiles = ((a.N + 255) / 256) * ((a.M + 255) / 256);
    if (pair_tiles >= sms / 2) return launch_pair<YT>(a, stream);
    int mc = 16;
    while (mc < 128 && mc < a.M) mc *= 2;
    const int64_t tiles = ((a.N + kRows - 1) / kRows) * ((a.M + mc - 1) / mc);
    const int splits = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, n_kt, sms / tiles})));
    switch (mc) {
        case 16: return launch_split<16, YT>(a, splits, stream);
        case 32: return launch_split<32, YT>(a, splits, stream);
        case 64: return launch_split<64, YT>(a, splits, stream);
        default: return launch_split<128, YT>(a, splits, stream);
    }
}

}  // namespace

cudaError_t launch_linear_i8(const LinearI8Args& a, cudaStream_t stream) {
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    return a.y_bf16 ? launch_typed<__nv_bfloat16>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace gdn
