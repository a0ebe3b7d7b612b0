// int8_kernels.cu -- rows quantised to 8-bit integers with a scale each (plain,
// or of silu(gate) * up), and the 8-bit product on the CUDA cores for few
// tokens.
#include <type_traits>

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
// it), as loaded.  VEC: the row is 16-byte aligned, k a multiple of 8.
template <typename T>
struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ float at(int i) const { return to_f32<T>(reinterpret_cast<const T*>(u)[i]); }
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load8(const T* row, int k, int K)
{
    Raw8<T> v;
    if (VEC && k + 8 <= K) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(T) / 2; ++i)
            v.u[i] = reinterpret_cast<const uint4*>(row + k)[i];
    } else {
        T* e = reinterpret_cast<T*>(v.u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = k + i < K ? row[k + i] : from_f32<T>(0.f);
    }
    return v;
}

// silu(g) * u.  The hardware exponential and divide are within a few ulp, far
// below the quantisation step that follows.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// What a thread keeps of eight elements between the two passes over its row: the
// 16-bit values as loaded, or fp32 values.
template <typename T, bool VEC, bool SILU>
struct Chunk8 {
    using E = typename std::conditional<SILU, float, T>::type;
    Raw8<E> v;
    __device__ __forceinline__ void load(const T* row, int k, int K)
    {
        if constexpr (SILU) {
            const Raw8<T> g = load8<T, VEC>(row, k, K), u = load8<T, VEC>(row + K, k, K);
            float* e = reinterpret_cast<float*>(v.u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = silu_mul(g.at(i), u.at(i));
        } else {
            v = load8<T, VEC>(row, k, K);
        }
    }
    // Largest magnitude so far, as bits: of a float, or two 16-bit floats side by
    // side.  On the bits, NaN > inf > every finite value.
    __device__ __forceinline__ uint32_t max_bits(uint32_t m) const
    {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v.u);
#pragma unroll
        for (unsigned i = 0; i < 2 * sizeof(E); ++i)
            m = sizeof(E) == 4 ? max(m, w[i] & 0x7fffffffu) : __vmaxu2(m, w[i] & 0x7fff7fffu);
        return m;
    }
    // ... as the bits of one float
    static __device__ __forceinline__ uint32_t as_f32_bits(uint32_t m)
    {
        if constexpr (sizeof(E) == 4) {
            return m;
        } else {
            const uint16_t h = static_cast<uint16_t>(max(m & 0xffffu, m >> 16));
            return __float_as_uint(to_f32<E>(*reinterpret_cast<const E*>(&h))) & 0x7fffffffu;
        }
    }
};

// rint(p) + 1.5 * 2^23 for |p| <= 127: the low byte of its bits is the code (ties
// to even, as the addition rounds)
constexpr float kRint = 12582912.0f;

// One block per row: the largest magnitude m, then q = rint(x * (127 * (1 / m)))
// and scale = m / 127.  A thread keeps up to NC chunks of 8 elements in registers,
// so that rows of up to 8 * NC * threads elements are read once; what lies
// beyond is read again.  A row with an inf or a NaN gets codes 0 and the scale
// NaN, which its products carry on.  Bound by its bytes: 16-bit values stay
// packed for the maximum (two a step), and the codes are rounded by an addition
// instead of a conversion (16 a clock and SM).
template <typename T, bool VEC, bool SILU, int NC>
__global__ void __launch_bounds__(1024) int8_quantize_kernel(QuantArgs a)
{
    using C = Chunk8<T, VEC, SILU>;
    __shared__ uint32_t part[32];
    pdl_wait();
    pdl_launch_dependents();
    if (a.err && blockIdx.x == 0 && threadIdx.x == 0)
        *a.err = 0;
    const int nt = blockDim.x, tid = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const T* row = static_cast<const T*>(a.x) + t * a.ld_x;
        C v[NC];
        uint32_t m = 0u;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = 8 * (tid + c * nt);
            if (k < a.K)
                v[c].load(row, k, a.K);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (8 * (tid + c * nt) < a.K)
                m = v[c].max_bits(m);
        for (int k = 8 * (tid + NC * nt); k < a.K; k += 8 * nt) {
            C u;
            u.load(row, k, a.K);
            m = u.max_bits(m);
        }
        m = __reduce_max_sync(kFull, C::as_f32_bits(m));
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
        __half* q16 = a.q16 + t * a.ld_q;
        auto store8 = [&](int k, const C& x) {
            float r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = inv != 0.f ? __fadd_rn(__fmul_rn(x.v.at(i), inv), kRint) : kRint;
            if (a.q16) {
                __half2 h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[i] = __floats2half2_rn(r[2 * i] - kRint, r[2 * i + 1] - kRint);
                if (k + 8 <= a.K) {
                    *reinterpret_cast<uint4*>(q16 + k) = *reinterpret_cast<const uint4*>(h);
                } else {
                    for (int i = 0; k + i < a.K; ++i)
                        q16[k + i] = __float2half_rn(r[i] - kRint);
                }
                return;
            }
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = __float_as_uint(r[i]);
            if (k + 8 <= a.K) {
                *reinterpret_cast<uint2*>(q + k) =
                    make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x40), __byte_perm(w[2], w[3], 0x40), 0x5410),
                               __byte_perm(__byte_perm(w[4], w[5], 0x40), __byte_perm(w[6], w[7], 0x40), 0x5410));
            } else {
                for (int i = 0; k + i < a.K; ++i)
                    q[k + i] = static_cast<int8_t>(w[i]);
            }
        };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = 8 * (tid + c * nt);
            if (k < a.K)
                store8(k, v[c]);
        }
        for (int k = 8 * (tid + NC * nt); k < a.K; k += 8 * nt) {
            C u;
            u.load(row, k, a.K);
            store8(k, u);
        }
    }
}

// 16 codes per thread
__global__ void __launch_bounds__(256)
    int8_to_f16_kernel(const int8_t* a, int64_t ld_a, int64_t T, int K, __half* out, int64_t ld_out, int* err)
{
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *err = 0;
    const int pieces = (K + 15) / 16;
    const int64_t total = T * pieces, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t t = i / pieces;
        const int k = static_cast<int>(i - t * pieces) * 16;
        __half h[16];
        if (k + 16 <= K) {
            union {
                uint4 u;
                int8_t c[16];
            } v;
            v.u = *reinterpret_cast<const uint4*>(a + t * ld_a + k);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                h[j] = __short2half_rn(v.c[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                h[j] = k + j < K ? __short2half_rn(a[t * ld_a + k + j]) : __half(0.f);
        }
        uint4* dst = reinterpret_cast<uint4*>(out + t * ld_out + k);
        dst[0] = reinterpret_cast<const uint4*>(h)[0];
        dst[1] = reinterpret_cast<const uint4*>(h)[1];
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
    if (a.err && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
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
    // chunks a thread keeps: 8 of 16-bit values, 4 of fp32 ones (32 registers)
    constexpr int NC = sizeof(T) == 2 && !SILU ? 8 : 4;
    const int chunks = (a.K + 7) / 8;
    // few rows: a chunk per thread, for latency; many: as many as it keeps
    int threads = a.T <= 2 * static_cast<int64_t>(sms) ? chunks : (chunks + NC - 1) / NC;
    threads = (threads + 31) / 32 * 32;
    threads = threads < 64 ? 64 : threads > 1024 ? 1024 : threads;
    const int grid = static_cast<int>(a.T < (1 << 30) ? a.T : (1 << 30));
    if (vec)
        return launch_pdl(int8_quantize_kernel<T, true, SILU, NC>, grid, threads, 0, s, a);
    return launch_pdl(int8_quantize_kernel<T, false, SILU, NC>, grid, threads, 0, s, a);
}

}  // namespace

cudaError_t launch_int8_quantize(const QuantArgs& a, int sms, cudaStream_t s)
{
    return with_type(a.type, [&](auto v) {
        return a.silu_mul ? launch_quantize_type<decltype(v), true>(a, sms, s)
                          : launch_quantize_type<decltype(v), false>(a, sms, s);
    });
}

cudaError_t launch_int8_to_f16(const int8_t* a, int64_t ld_a, int64_t T, int K, __half* out, int64_t ld_out,
                               int* err, int sms, cudaStream_t s)
{
    const int64_t blocks = (T * ((K + 15) / 16) + 255) / 256, most = 8 * static_cast<int64_t>(sms);
    return launch_pdl(int8_to_f16_kernel, static_cast<int>(blocks < most ? blocks : most), 256, 0, s, a, ld_a, T, K,
                      out, ld_out, err);
}

cudaError_t launch_int8_rows(const Int8Args& a, int sms, cudaStream_t s)
{
    return with_type(a.type, [&](auto v) { return launch_rows_type<decltype(v)>(a, sms, s); });
}

}  // namespace chord
