// int8_gemm.cu -- the 8-bit product on the 5th-generation tensor cores.
//
// This part's 8-bit integer tensor rate is a small fraction of its 16-bit one
// and tcgen05 has no integer kind here, so the codes enter the MMA as fp16,
// which holds every 8-bit integer exactly.  A product of two codes is an
// integer of at most 2^14, and a chain of 1024 of them stays an integer of at
// most 2^24, which fp32 holds exactly in whatever order the tensor core adds.
// Chains of 1024 (kChain K stages) alternate between two accumulators in tensor
// memory; the epilogue warps add each finished one into 32-bit integers in
// registers, so the sum over any K is the exact integer.
//
// D[128 channels, NT tokens] = W_tile[128, K] A_tile[NT, K]^T: the weight is the
// M operand, converted into tensor memory, the tokens the N operand, converted
// into shared memory.  Both arrive as raw 8-bit boxes by TMA, half the bytes of
// a 16-bit operand, and are converted once per stage:
//   warp 0       producer: one box of each operand per K stage of 128 codes
//   warp 1       MMA issuer;  warp 2  owner of the tensor memory
//   warps 4-11   converters, two per lane quadrant: code ^ 0x80 under the fp16
//                exponent of 1024 is 1024 + 128 + code; subtracting 1152 is exact
//                (1.25 instructions per code)
//   warps 12-19  epilogue, two per lane quadrant (a half of the token columns each)
// Split K: a weight with fewer tiles than SMs is cut along K over the CTAs of a
// cluster; the integer partial sums meet in distributed shared memory.
// Every wait is bounded (2 s): on expiry CHORD_DEVERR_TIMEOUT is recorded, every
// role leaves its loop and tensor memory is freed.
#include <cudaTypedefs.h>

#include "block_kernels.h"
#include "device.cuh"

namespace chord {

namespace {

constexpr int kBK = 128;     // codes of a K stage (one 128-byte swizzled row)
constexpr int kChain = 8;    // K stages of an accumulation chain (1024 products)
constexpr int kTileM = 128;  // channels of a tile
constexpr int kConvWarps = 8;
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 12;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);

struct Int8Gemm {
    Int8Args p;
    int nt;        // token tile: a multiple of 16, at most NTMAX
    int n_tiles;   // channel tiles
    int units;     // channel tiles * token tiles
    int split;     // CTAs of a cluster that share a unit along K
    int w_ready;   // the weight may be read before the preceding kernel has ended
};

template <int NTMAX_, int RS_, int AS_>
struct Int8Cfg {
    static constexpr int NTMAX = NTMAX_;  // largest token tile
    static constexpr int RS = RS_;        // raw stages in shared memory
    static constexpr int AS = AS_;        // converted stages (TMEM and shared memory)
    static constexpr int W_RAW = kTileM * kBK;
    static constexpr int T_RAW = NTMAX * kBK;
    static constexpr int B_REGION = NTMAX * 128;  // one 64-element column block of the tokens
    static constexpr int B_STAGE = 2 * B_REGION;
    static constexpr int OFF_W = 0;
    static constexpr int OFF_T = OFF_W + RS * W_RAW;
    static constexpr int OFF_B = OFF_T + RS * T_RAW;
    static constexpr int OFF_BARS = OFF_B + AS * B_STAGE;
    static constexpr int NBARS = 2 * RS + 2 * AS + 4 + 1;
    static constexpr int OFF_MISC = OFF_BARS + 8 * NBARS;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;  // + alignment slack
    static constexpr int A_COLS = kBK / 2;
    static constexpr int D_COL0 = AS * A_COLS;
    static constexpr int TMEM_COLS = 512;
    static_assert(NTMAX % 16 == 0 && NTMAX <= 256, "token tile");
    static_assert(T_RAW % 1024 == 0, "swizzle atoms need 1024-byte alignment");
    static_assert(D_COL0 + 2 * NTMAX <= TMEM_COLS, "tensor memory budget");
    static_assert(SMEM <= 232448 && SMEM > 116 * 1024, "one CTA per SM");
    // (split K: the partial sums take the place of the raw stages)
    static_assert(kTileM * NTMAX * 4 <= OFF_BARS, "partial sums");
};

// four 8-bit codes -> four fp16 (two registers), exact
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 base = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), base);
    const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), base);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N)
{
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                   "=r"(v[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr, uint32_t rank)
{
    uint32_t ra;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}

// out (one type) of one token and channel
template <typename T>
__device__ __forceinline__ void store_sum(const Int8Args& a, int64_t t, int n, int sum, float ws)
{
    float v = static_cast<float>(sum) * a.a_scale[t] * ws;
    if (a.residual)
        v += to_f32<T>(static_cast<const T*>(a.residual)[t * a.ld_r + n]);
    static_cast<T*>(a.out)[t * a.ld_out + n] = from_f32<T>(v);
}

template <class C, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap t_map,
                     const Int8Gemm g)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - raw_u32);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = g.split > 1 ? static_cast<int>(cluster_rank()) : 0;

    const uint32_t bar0 = sbase + C::OFF_BARS;
    auto raw_full = [&](int s) { return bar0 + 8u * s; };
    auto raw_empty = [&](int s) { return bar0 + 8u * (C::RS + s); };
    auto cv_full = [&](int s) { return bar0 + 8u * (2 * C::RS + s); };
    auto cv_empty = [&](int s) { return bar0 + 8u * (2 * C::RS + C::AS + s); };
    auto acc_full = [&](int s) { return bar0 + 8u * (2 * C::RS + 2 * C::AS + s); };
    auto acc_empty = [&](int s) { return bar0 + 8u * (2 * C::RS + 2 * C::AS + 2 + s); };
    const uint32_t drain_bar = bar0 + 8u * (C::NBARS - 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    int* err = g.p.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::RS; ++s) {
            mbar_init(raw_full(s), 1);
            mbar_init(raw_empty(s), kConvWarps);
        }
        for (int s = 0; s < C::AS; ++s) {
            mbar_init(cv_full(s), kConvWarps);
            mbar_init(cv_empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full(s), 1);
            mbar_init(acc_empty(s), kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_fence_init();
        prefetch_tensormap(&w_map);
        prefetch_tensormap(&t_map);
    }
    if (warp == 2)
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (!g.w_ready)
        pdl_wait();
    pdl_launch_dependents();
    if (g.p.clear_err && blockIdx.x == 0 && threadIdx.x == 0)
        *err = 0;  // (a wait that expires sets it 2 s from now at the earliest)

    const int KT = (g.p.K + kBK - 1) / kBK;
    const int k0 = rank * KT / g.split, k1 = (rank + 1) * KT / g.split;  // this CTA's K stages
    const int u0 = blockIdx.x / g.split, ustep = gridDim.x / g.split;
    const int nt = g.nt;
    int issued = 0;  // raw stages whose copies were issued

    if (warp == 0) {
        // ------------------------------------------------------------- producer
        const uint64_t pol_w = g.units > g.n_tiles ? policy_evict_last() : policy_evict_first();
        const uint64_t pol_t = policy_evict_last();
        const uint32_t bytes = C::W_RAW + nt * kBK;
        bool ok = true;
        // the weight boxes of the first stages go out while the preceding kernel
        // still writes the tokens
        int early = 0;
        if (g.w_ready) {
            if (u0 < g.units)
                for (; early < C::RS && k0 + early < k1; ++early)
                    if (lane == 0) {
                        mbar_arrive_expect_tx(raw_full(early), bytes);
                        tma_load_2d(sbase + C::OFF_W + early * C::W_RAW, &w_map, (k0 + early) * kBK,
                                    u0 % g.n_tiles * kTileM, raw_full(early), pol_w);
                    }
            pdl_wait();
        }
        int it = 0;
        for (int u = u0; u < g.units && ok; u += ustep) {
            const int row_w = u % g.n_tiles * kTileM, row_t = u / g.n_tiles * nt;
            for (int ks = k0; ks < k1; ++ks, ++it) {
                const int s = it % C::RS;
                if (!mbar_wait(raw_empty(s), ((it / C::RS) & 1) ^ 1, abort_flag, err)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (it >= early) {
                        mbar_arrive_expect_tx(raw_full(s), bytes);
                        tma_load_2d(sbase + C::OFF_W + s * C::W_RAW, &w_map, ks * kBK, row_w, raw_full(s), pol_w);
                    }
                    tma_load_2d(sbase + C::OFF_T + s * C::T_RAW, &t_map, ks * kBK, row_t, raw_full(s), pol_t);
                }
                __syncwarp();
            }
        }
        issued = it > early ? it : early;
    } else if (warp == 1) {
        // ----------------------------------------------------------- MMA issuer
        const uint32_t idesc = idesc_f16_f32(kTileM, nt);
        int it = 0, pc = 0, any = 0;
        bool ok = true;
        for (int u = u0; u < g.units && ok; u += ustep) {
            for (int c0 = k0; c0 < k1 && ok; c0 += kChain, ++pc) {
                const int c1 = c0 + kChain < k1 ? c0 + kChain : k1;
                const int acc = pc & 1;
                if (!__all_sync(0xffffffffu, mbar_wait(acc_empty(acc), ((pc >> 1) & 1) ^ 1, abort_flag, err))) {
                    ok = false;
                    break;
                }
                for (int ks = c0; ks < c1; ++ks, ++it) {
                    const int s = it % C::AS;
                    if (!__all_sync(0xffffffffu, mbar_wait(cv_full(s), (it / C::AS) & 1, abort_flag, err))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_stage8<C::B_REGION / 16>(tmem + C::D_COL0 + acc * C::NTMAX, tmem + s * C::A_COLS,
                                                 smem_desc_sw128(sbase + C::OFF_B + s * C::B_STAGE), idesc,
                                                 ks != c0 ? 1u : 0u);
                    any = 1;
                    mma_commit_elect(cv_empty(s));
                }
                if (ok)
                    mma_commit_elect(acc_full(acc));
            }
        }
        if (!ok && any) {  // work in flight ends before tensor memory is freed
            mma_commit_elect(drain_bar);
            mbar_drain(drain_bar, 0);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < kEpiWarp0) {
        // ------------------------------------------------------------ converters
        const int cw = warp - 4, half = cw >> 2, q = warp & 3;
        const int row = q * 32 + lane;
        const int tid = threadIdx.x - 128;  // 0..255
        const uint32_t tlane = static_cast<uint32_t>(q * 32) << 16;
        const int pieces = nt * 8;  // 16-byte pieces of a token stage
        int it = 0;
        bool ok = true;
        for (int u = u0; u < g.units && ok; u += ustep) {
            for (int ks = k0; ks < k1; ++ks, ++it) {
                const int rs = it % C::RS, s = it % C::AS;
                if (!mbar_wait(raw_full(rs), (it / C::RS) & 1, abort_flag, err) ||
                    !mbar_wait(cv_empty(s), ((it / C::AS) & 1) ^ 1, abort_flag, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // 64 codes of one channel -> 32 TMEM columns of this lane
                const uint8_t* wrow = smem + C::OFF_W + rs * C::W_RAW + row * 128;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t o[16];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            wrow + (((half * 4 + p * 2 + c) ^ (row & 7)) << 4));
                        codes_to_f16(v.x, o[8 * c], o[8 * c + 1]);
                        codes_to_f16(v.y, o[8 * c + 2], o[8 * c + 3]);
                        codes_to_f16(v.z, o[8 * c + 4], o[8 * c + 5]);
                        codes_to_f16(v.w, o[8 * c + 6], o[8 * c + 7]);
                    }
                    tmem_st_x16(tmem + tlane + s * C::A_COLS + half * 32 + p * 16, o);
                }
                // tokens: piece c of row r (16 codes) becomes two 16-byte pieces of the
                // 128-byte swizzled fp16 row; lanes of the upper half write theirs in
                // the other order, so that eight lanes cover all banks
                const uint8_t* traw = smem + C::OFF_T + rs * C::T_RAW;
                uint8_t* tb = smem + C::OFF_B + s * C::B_STAGE;
#pragma unroll 2
                for (int i = tid; i < pieces; i += 256) {
                    const int r = i >> 3, c = i & 7;
                    const uint4 v = *reinterpret_cast<const uint4*>(traw + r * 128 + ((c ^ (r & 7)) << 4));
                    uint4 a, b;
                    codes_to_f16(v.x, a.x, a.y);
                    codes_to_f16(v.y, a.z, a.w);
                    codes_to_f16(v.z, b.x, b.y);
                    codes_to_f16(v.w, b.z, b.w);
                    uint8_t* dst = tb + (c >> 2) * C::B_REGION + r * 128;
                    const int p0 = ((c & 3) * 2) ^ (r & 7), sw = c >> 2;
                    *reinterpret_cast<uint4*>(dst + ((p0 ^ sw) << 4)) = sw ? b : a;
                    *reinterpret_cast<uint4*>(dst + ((p0 ^ sw ^ 1) << 4)) = sw ? a : b;
                }
                // reads of the raw stage before the next TMA into it, writes of the
                // token stage before the MMA reads it
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(raw_empty(rs));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(cv_full(s));
            }
        }
    } else if (warp >= kEpiWarp0) {
        // -------------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
        const uint32_t tlane = static_cast<uint32_t>(q * 32) << 16;
        const int ncol = nt / 2, col0 = half * ncol;  // (nt % 16 == 0: ncol % 8 == 0)
        if (g.w_ready)
            pdl_wait();  // (a_scale, residual)
        int pc = 0;
        bool ok = true;
        for (int u = u0; u < g.units && ok; u += ustep) {
            int sum[C::NTMAX / 2];
            for (int c0 = k0; c0 < k1; c0 += kChain, ++pc) {
                const int acc = pc & 1;
                if (!mbar_wait(acc_full(acc), (pc >> 1) & 1, abort_flag, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool first = c0 == k0;
#pragma unroll
                for (int j = 0; j < C::NTMAX / 2; j += 8) {
                    if (j < ncol) {
                        uint32_t v[8];
                        tmem_ld_x8(tmem + tlane + C::D_COL0 + acc * C::NTMAX + col0 + j, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int x = __float2int_rn(__uint_as_float(v[i]));
                            sum[j + i] = first ? x : sum[j + i] + x;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(acc_empty(acc));
            }
            if (!ok)
                break;
            const int r = q * 32 + lane;
            if (g.split > 1) {
                // (this CTA's only unit: its raw stages have all been converted)
                int* part = reinterpret_cast<int*>(smem);
#pragma unroll
                for (int j = 0; j < C::NTMAX / 2; ++j)
                    if (j < ncol)
                        part[(col0 + j) * kTileM + r] = sum[j];
            } else {
                const int n = u % g.n_tiles * kTileM + r;
                const int64_t t0 = static_cast<int64_t>(u / g.n_tiles) * nt + col0;
                if (n < g.p.N) {
                    const float ws = g.p.w_scale[n];
#pragma unroll
                    for (int j = 0; j < C::NTMAX / 2; ++j)
                        if (j < ncol && t0 + j < g.p.T)
                            store_sum<T>(g.p, t0 + j, n, sum[j], ws);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 0) {
        // copies issued but never consumed land before the CTA ends
        if (lane == 0)
            for (int i = issued > C::RS ? issued - C::RS : 0; i < issued; ++i)
                mbar_drain(raw_full(i % C::RS), (i / C::RS) & 1);
        __syncwarp();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (g.split > 1) {
        // every CTA of the cluster finishes a share of the token columns
        __syncthreads();
        cluster_sync_all();
        pdl_wait();
        const int u = u0;
        const int n0 = u % g.n_tiles * kTileM;
        const int64_t t0 = static_cast<int64_t>(u / g.n_tiles) * nt;
        const int c0 = rank * nt / g.split, c1 = (rank + 1) * nt / g.split;
        for (int i = threadIdx.x; i < (c1 - c0) * kTileM; i += kThreads) {
            const int col = c0 + i / kTileM, r = i % kTileM;
            const uint32_t at = sbase + 4u * (col * kTileM + r);
            int sum = 0;
            for (int k = 0; k < g.split; ++k)
                sum += ld_cluster_s32(at, k);
            if (n0 + r < g.p.N && t0 + col < g.p.T)
                store_sum<T>(g.p, t0 + col, n0 + r, sum, g.p.w_scale[n0 + r]);
        }
        cluster_sync_all();  // (the partial sums stay until every CTA has read them)
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 f = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    return f;
}

// Rows of 8-bit codes: boxes of `rows` rows x 128 codes, 128-byte swizzle, zero
// past the last row and past code K of a row.
cudaError_t codes_rows_map(const int8_t* p, int64_t n, int K, int64_t ld, int rows, CUtensorMap* out)
{
    const auto encode = encoder();
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(n)};
    // (a single row has no distance: any multiple of 16 will do)
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld >= K ? ld : (K + 15) / 16 * 16)};
    const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(rows)}, es[2] = {1, 1};
    return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <class C, typename T>
cudaError_t launch_cfg(Int8Gemm g, int sms, cudaStream_t s)
{
    static bool attr_set[64] = {};  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(int8_gemm_kernel<C, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess)
            return e;
        attr_set[dev] = true;
    }
    CUtensorMap wm, tm;
    if ((e = codes_rows_map(g.p.w, g.p.N, g.p.K, g.p.ld_w, kTileM, &wm)) != cudaSuccess ||
        (e = codes_rows_map(g.p.a, g.p.T, g.p.K, g.p.ld_a, g.nt, &tm)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = g.split > 1 ? g.units * g.split : (g.units < sms ? g.units : sms);
    cfg.blockDim = kThreads;
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = g_launch_pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = g.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, int8_gemm_kernel<C, T>, wm, tm, g);
}

using CfgT32 = Int8Cfg<32, 8, 4>;
using CfgT128 = Int8Cfg<128, 4, 2>;
using CfgT192 = Int8Cfg<192, 3, 2>;

template <typename T>
cudaError_t launch_type(const Int8Args& a, int w_ready, int sms, cudaStream_t s)
{
    Int8Gemm g{};
    g.p = a;
    g.w_ready = w_ready;
    g.n_tiles = (a.N + kTileM - 1) / kTileM;
    // token tile: the whole batch where it fits one, else the width of 128..192
    // whose rounds of units cost least
    const int64_t t16 = (a.T + 15) / 16 * 16;
    if (t16 <= 192) {
        g.nt = static_cast<int>(t16);
    } else {
        int64_t best = INT64_MAX;
        for (int nt = 192; nt >= 128; nt -= 16) {
            const int64_t units = (a.T + nt - 1) / nt * g.n_tiles;
            const int64_t cost = (units + sms - 1) / sms * (nt + 16);
            if (cost < best) {
                best = cost;
                g.nt = nt;
            }
        }
    }
    const int64_t units = (a.T + g.nt - 1) / g.nt * g.n_tiles;
    if (units > INT32_MAX)
        return cudaErrorInvalidValue;
    g.units = static_cast<int>(units);
    const int KT = (a.K + kBK - 1) / kBK;
    g.split = 1;
    while (g.split < 8 && g.units * g.split * 2 <= sms && KT >= 4 * g.split)
        g.split *= 2;
    if (g.nt <= 32)
        return launch_cfg<CfgT32, T>(g, sms, s);
    if (g.nt <= 128)
        return launch_cfg<CfgT128, T>(g, sms, s);
    return launch_cfg<CfgT192, T>(g, sms, s);
}

}  // namespace

cudaError_t launch_int8_gemm(const Int8Args& a, int w_ready, int sms, cudaStream_t s)
{
    return with_type(a.type, [&](auto v) { return launch_type<decltype(v)>(a, w_ready, sms, s); });
}

}  // namespace chord
