// int8_kernels.cu -- rows quantised to 8-bit integers with a scale each (plain,
// or of silu(gate) * up), and the 8-bit product on the CUDA cores for few
// tokens.
#include "block_kernels.h"
#include "device.cuh"

namespace chord {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kInfBits = 0x7f800000u;
// rows whose largest magnitude is below 2^-100 count as zero: 127 * (1 / m) would
// leave fp32's range for the smallest of them
constexpr uint32_t kTinyBits = (127u - 100u) << 23;

// Eight consecutive elements of a row from element k (fewer at its end, 0 past
// it).  VEC: the row is 16-byte aligned, k a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int k, int K, float (&v)[8])
{
    if (VEC && k + 8 <= K) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4*>(row + k);
            const float4 b = *reinterpret_cast<const float4*>(row + k + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            union {
                uint4 u;
                T e[8];
            } p;
            p.u = *reinterpret_cast<const uint4*>(row + k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = to_f32<T>(p.e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = k + i < K ? to_f32<T>(row[k + i]) : 0.f;
    }
}

// silu(g) * u.  The hardware exponential and divide are within a few ulp, far
// below the quantisation step that follows.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

template <typename T, bool VEC, bool SILU>
__device__ __forceinline__ void load8_value(const T* row, int k, int K, float (&v)[8])
{
    load8<T, VEC>(row, k, K, v);
    if constexpr (SILU) {
        float u[8];
        load8<T, VEC>(row + K, k, K, u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = silu_mul(v[i], u[i]);
    }
}

// One block per row: the largest magnitude m, then q = rint(x * (127 * (1 / m)))
// and scale = m / 127.  A thread holds up to NC chunks of 8 elements in registers,
// so that rows of up to 8 * NC * threads elements are read once; what lies
// beyond is read again.  m is taken on the bit patterns, where NaN > inf > every
// finite value: such a row gets codes 0 and the scale NaN, which its products
// carry on.
template <typename T, bool VEC, bool SILU, int NC>
__global__ void __launch_bounds__(1024) int8_quantize_kernel(QuantArgs a)
{
    __shared__ uint32_t part[32];
    pdl_wait();
    pdl_launch_dependents();
    if (a.err && blockIdx.x == 0 && threadIdx.x == 0)
        *a.err = 0;
    const int nt = blockDim.x, tid = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const T* row = static_cast<const T*>(a.x) + t * a.ld_x;
        float v[NC][8];
        uint32_t m = 0u;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = 8 * (tid + c * nt);
            if (k < a.K) {
                load8_value<T, VEC, SILU>(row, k, a.K, v[c]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    m = max(m, __float_as_uint(v[c][i]) & 0x7fffffffu);
            }
        }
        for (int k = 8 * (tid + NC * nt); k < a.K; k += 8 * nt) {
            float u[8];
            load8_value<T, VEC, SILU>(row, k, a.K, u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = max(m, __float_as_uint(u[i]) & 0x7fffffffu);
        }
        m = __reduce_max_sync(kFull, m);
        if ((tid & 31) == 0)
            part[tid >> 5] = m;
        __syncthreads();
        m = __reduce_max_sync(kFull, (tid & 31) < (nt >> 5) ? part[tid & 31] : 0u);
        __syncthreads();  // (part is written again for the next row)
        const float top = __uint_as_float(m);
        float inv = 0.f, scale = 0.f;
        if (m >= kInfBits)
            scale = __uint_as_float(0x7fffffffu);
        else if (m >= kTinyBits) {
            inv = 127.0f * (1.0f / top);
            scale = top / 127.0f;
        }
        if (tid == 0)
            a.scale[t] = scale;
        int8_t* q = a.q + t * a.ld_q;
        auto store8 = [&](int k, const float (&x)[8]) {
            uint32_t w[2] = {0u, 0u};
            if (inv != 0.f) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i >> 2] |= (static_cast<uint32_t>(__float2int_rn(x[i] * inv)) & 0xffu) << (8 * (i & 3));
            }
            if (k + 8 <= a.K) {
                *reinterpret_cast<uint2*>(q + k) = make_uint2(w[0], w[1]);
            } else {
                for (int i = 0; k + i < a.K; ++i)
                    q[k + i] = static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)));
            }
        };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = 8 * (tid + c * nt);
            if (k < a.K)
                store8(k, v[c]);
        }
        for (int k = 8 * (tid + NC * nt); k < a.K; k += 8 * nt) {
            float u[8];
            load8_value<T, VEC, SILU>(row, k, a.K, u);
            store8(k, u);
        }
    }
}

// ---------------------------------------------------------------------------
// the product on the CUDA cores: dp4a, exact in 32-bit integers
// ---------------------------------------------------------------------------
constexpr int kRowsN = 2;  // channels per warp

// 16 codes of a row from k; past K (only the last chunk of a row) zero.  A chunk
// is never read past the row's K codes: the row may end its allocation.
__device__ __forceinline__ int4 load_codes(const int8_t* row, int k, int K)
{
    if (k + 16 <= K)
        return *reinterpret_cast<const int4*>(row + k);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K)
            w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + i])) << (8 * (i & 3));
    return make_int4(static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]),
                     static_cast<int>(w[3]));
}

template <typename T>
__device__ __forceinline__ void store_out(const Int8Args& a, int64_t t, int n, int sum)
{
    float v = static_cast<float>(sum) * a.a_scale[t] * a.w_scale[n];
    if (a.residual)
        v += to_f32<T>(static_cast<const T*>(a.residual)[t * a.ld_r + n]);
    static_cast<T*>(a.out)[t * a.ld_out + n] = from_f32<T>(v);
}

// A warp takes kRowsN channels and TT tokens; its lanes walk K in 16-byte
// chunks.  ks warps of a block share the channels, each a part of K, so that a
// narrow weight still keeps every SM's loads in flight; their integer partial
// sums are added in shared memory.
template <typename T, int TT>
__global__ void __launch_bounds__(256) int8_rows_kernel(Int8Args a, int ks)
{
    __shared__ int part[8][kRowsN * TT];
    pdl_launch_dependents();
    pdl_wait();
    if (a.err && a.clear_err && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *a.err = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = 8 / ks;
    const int n0 = (blockIdx.x * groups + warp / ks) * kRowsN;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * TT;
    int acc[kRowsN][TT] = {};
    const int8_t* wr[kRowsN];
#pragma unroll
    for (int r = 0; r < kRowsN; ++r)
        wr[r] = a.w + static_cast<int64_t>(min(n0 + r, a.N - 1)) * a.ld_w;
    if (n0 < a.N) {
#pragma unroll 4
        for (int k = 16 * (lane + 32 * (warp % ks)); k < a.K; k += 512 * ks) {
            int4 wv[kRowsN];
#pragma unroll
            for (int r = 0; r < kRowsN; ++r)
                wv[r] = load_codes(wr[r], k, a.K);
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                if (t0 + i < a.T) {
                    const int4 av = load_codes(a.a + (t0 + i) * a.ld_a, k, a.K);
#pragma unroll
                    for (int r = 0; r < kRowsN; ++r) {
                        acc[r][i] = __dp4a(wv[r].x, av.x, acc[r][i]);
                        acc[r][i] = __dp4a(wv[r].y, av.y, acc[r][i]);
                        acc[r][i] = __dp4a(wv[r].z, av.z, acc[r][i]);
                        acc[r][i] = __dp4a(wv[r].w, av.w, acc[r][i]);
                    }
                }
            }
        }
    }
    // lane r * TT + i keeps the sum of channel r and token i
    int mine = 0;
#pragma unroll
    for (int r = 0; r < kRowsN; ++r)
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int s = __reduce_add_sync(kFull, acc[r][i]);
            if (lane == r * TT + i)
                mine = s;
        }
    if (ks > 1) {
        if (lane < kRowsN * TT)
            part[warp][lane] = mine;
        __syncthreads();
        if (warp % ks != 0)
            return;
        if (lane < kRowsN * TT)
            for (int j = 1; j < ks; ++j)
                mine += part[warp + j][lane];
    }
    const int n = n0 + lane / TT;
    const int64_t t = t0 + lane % TT;
    if (lane < kRowsN * TT && n < a.N && t < a.T)
        store_out<T>(a, t, n, mine);
}

template <typename T>
cudaError_t launch_rows_type(const Int8Args& a, int sms, cudaStream_t s)
{
    // parts of K per channel pair: until 16 warps per SM have work, each part
    // at least one sweep of its lanes (512 codes)
    int ks = 1;
    const int64_t pairs = (a.N + kRowsN - 1) / kRowsN;
    while (ks < 8 && pairs * ks < 16 * static_cast<int64_t>(sms) && a.K > 512 * ks)
        ks *= 2;
    const int per_block = 8 / ks * kRowsN;
    const int tt = a.T >= 5 ? 8 : a.T >= 3 ? 4 : static_cast<int>(a.T);
    const int64_t ty = (a.T + tt - 1) / tt;
    for (int64_t y = 0; y < ty; y += 65535) {  // (the grid's y limit)
        Int8Args b = a;
        b.T = a.T - y * tt;
        if (b.T > 65535 * static_cast<int64_t>(tt))
            b.T = 65535 * static_cast<int64_t>(tt);
        b.a = a.a + y * tt * a.ld_a;
        b.a_scale = a.a_scale + y * tt;
        b.out = static_cast<T*>(a.out) + y * tt * a.ld_out;
        if (a.residual)
            b.residual = static_cast<const T*>(a.residual) + y * tt * a.ld_r;
        b.clear_err = a.clear_err && y == 0;
        const dim3 grid((a.N + per_block - 1) / per_block, static_cast<unsigned>((b.T + tt - 1) / tt));
        cudaError_t e;
        switch (tt) {
        case 1: e = launch_pdl(int8_rows_kernel<T, 1>, grid, 256, 0, s, b, ks); break;
        case 2: e = launch_pdl(int8_rows_kernel<T, 2>, grid, 256, 0, s, b, ks); break;
        case 4: e = launch_pdl(int8_rows_kernel<T, 4>, grid, 256, 0, s, b, ks); break;
        default: e = launch_pdl(int8_rows_kernel<T, 8>, grid, 256, 0, s, b, ks); break;
        }
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

template <typename T, bool SILU>
cudaError_t launch_quantize_type(const QuantArgs& a, int sms, cudaStream_t s)
{
    const int64_t row_bytes = a.ld_x * static_cast<int64_t>(sizeof(T));
    bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && row_bytes % 16 == 0;
    if (SILU)  // (the up half starts K elements into the row)
        vec = vec && a.K * static_cast<int64_t>(sizeof(T)) % 16 == 0;
    const int chunks = (a.K + 7) / 8;
    // few rows: a chunk per thread, for latency; many: up to four
    int threads = a.T <= 2 * static_cast<int64_t>(sms) ? chunks : (chunks + 3) / 4;
    threads = (threads + 31) / 32 * 32;
    threads = threads < 64 ? 64 : threads > 1024 ? 1024 : threads;
    const int grid = static_cast<int>(a.T < (1 << 30) ? a.T : (1 << 30));
    if (vec)
        return launch_pdl(int8_quantize_kernel<T, true, SILU, 4>, grid, threads, 0, s, a);
    return launch_pdl(int8_quantize_kernel<T, false, SILU, 4>, grid, threads, 0, s, a);
}

}  // namespace

cudaError_t launch_int8_quantize(const QuantArgs& a, int sms, cudaStream_t s)
{
    return with_type(a.type, [&](auto v) {
        return a.silu_mul ? launch_quantize_type<decltype(v), true>(a, sms, s)
                          : launch_quantize_type<decltype(v), false>(a, sms, s);
    });
}

cudaError_t launch_int8_rows(const Int8Args& a, int sms, cudaStream_t s)
{
    return with_type(a.type, [&](auto v) { return launch_rows_type<decltype(v)>(a, sms, s); });
}

}  // namespace chord
