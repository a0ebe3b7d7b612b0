// route_kernels.cu -- the scored router (softmax or sigmoid scores, a bias that
// steers the choice, expert groups, top-k, renormalised and scaled weights) and
// the gradient of its weights at the logits.
#include <cfloat>
#include <climits>

#include "block_kernels.h"
#include "device.cuh"

namespace chord {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// Order-preserving map of a float (no NaN, no -0) to uint32.  Selection works
// on these keys; two values below every real key mark what cannot be chosen:
// kKeyMasked (the key of -inf) a masked expert or one of a group left out,
// which only fills slots that nothing else can, and 0 a lane position past E
// or an expert already chosen.
constexpr uint32_t kKeyMasked = 0x007fffffu;

__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// A logit as the router sees it: NaN and -inf are masked (-inf), +inf counts
// as the largest finite float, -0 as 0.
template <typename T>
__device__ __forceinline__ float load_logit(const T* p)
{
    const float v = to_f32<T>(*p);
    return v == v ? fminf(v, FLT_MAX) + 0.f : -INFINITY;
}

__device__ __forceinline__ float warp_max(float v)
{
    return order_value(__reduce_max_sync(kFull, order_key(v)));
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + expf(-x)); }

// Bit set of the topk_group groups with the largest scores (ties to the lower
// group).  vals: the warp's experts' values in shared memory, -inf where
// masked; 32 / pow2(n_group) lanes walk each group for its two largest values.
__device__ uint32_t choose_groups(const float* vals, const MoeRouteArgs& a, int size, int lane)
{
    int lanes = 32;  // lanes per group, a power of two
    while (lanes * a.n_group > 32)
        lanes >>= 1;
    const int g = lane / lanes, sub = lane % lanes;
    float a1 = -INFINITY, a2 = -INFINITY;
    if (g < a.n_group) {
        for (int m = sub; m < size; m += lanes) {
            const float v = vals[g * size + m];
            a2 = fmaxf(a2, fminf(a1, v));
            a1 = fmaxf(a1, v);
        }
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        const float b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
        a2 = fmaxf(fmaxf(a2, b2), fminf(a1, b1));
        a1 = fmaxf(a1, b1);
    }
    const float score = (a.group_top == 1 || a2 == -INFINITY) ? a1 : a1 + a2;
    uint32_t key = (g < a.n_group && sub == 0) ? order_key(score + 0.f) : 0u;
    uint32_t kept = 0u;
    for (int j = 0; j < a.topk_group; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, key);
        const int w = __ffs(__ballot_sync(kFull, key == top)) - 1;
        kept |= 1u << (w / lanes);
        if (lane == w)
            key = 0u;
    }
    return kept;
}

// One warp routes one token; lane l holds experts l, l + 32, ... (NI of them).
// k rounds pick the largest key and, among equal keys, the lowest expert: each
// lane keeps its own best, two warp reductions find the winner, and only then
// the winner's lane looks for its next best.
template <typename TL, int NI>
__device__ void route_token(const MoeRouteArgs& a, int64_t t, int lane, float* vals)
{
    const TL* row = static_cast<const TL*>(a.logits) + t * a.ld;
    const bool sigmoid = a.scoring == CHORD_SCORE_SIGMOID;
    float x[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < a.E ? load_logit(row + e) : -INFINITY;
    }
    float top = 0.f, sum = 1.f;  // softmax: largest logit, sum of exponentials
    if (!sigmoid) {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < NI; ++i)
            m = fmaxf(m, x[i]);
        top = warp_max(m);
        if (top == -INFINITY)
            top = 0.f;  // every expert is masked: every exponential is 0
        if (a.bias || !a.renorm) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                sum += expf(x[i] - top);
            sum = warp_sum(sum);
        }
    }
    // keys: score + bias, or without a bias the logits, whose order is that of
    // the scores; groups are ranked by score + bias (without a bias by the
    // scores, for softmax before the division by their sum)
    uint32_t key[NI];
    if (a.bias || a.n_group > 1) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            const bool real = x[i] != -INFINITY;
            float v = -INFINITY;
            if (real) {
                v = sigmoid ? sigmoid_f32(x[i]) : expf(x[i] - top);
                if (a.bias) {
                    v = (sigmoid ? v : v / sum) + a.bias[e] + 0.f;
                    v = v == v ? v : -INFINITY;  // (a NaN bias masks its expert)
                }
            }
            if (e < a.E && a.n_group > 1)
                vals[e] = v;
            key[i] = e >= a.E ? 0u : !real ? kKeyMasked : order_key(a.bias ? v : x[i]);
        }
        if (a.n_group > 1) {
            const int size = a.E / a.n_group;
            __syncwarp();
            const uint32_t kept = choose_groups(vals, a, size, lane);
            __syncwarp();
            // e / size for e < 1024: e * ceil(2^20 / size) >> 20 is exact
            const uint32_t magic = ((1u << 20) + size - 1) / size;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const uint32_t e = lane + 32 * i;
                if (key[i] != 0u && !((kept >> ((e * magic) >> 20)) & 1u))
                    key[i] = kKeyMasked;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            key[i] = lane + 32 * i >= a.E ? 0u : order_key(x[i]);
    }

    int my_id = 0;          // lane j keeps the j-th choice
    uint32_t my_key = 0u;
    uint32_t best = 0u;     // this lane's largest key and its lowest expert
    int best_e = 0;
    auto refresh = [&]() {
        best = key[0];
#pragma unroll
        for (int i = 1; i < NI; ++i)
            best = max(best, key[i]);
#pragma unroll
        for (int i = NI - 1; i >= 0; --i)
            if (key[i] == best)
                best_e = lane + 32 * i;
    };
    refresh();
    for (int j = 0; j < a.k; ++j) {
        const uint32_t m = __reduce_max_sync(kFull, best);
        const int e = __reduce_min_sync(kFull, best == m ? best_e : INT_MAX);
        if (lane == j) {
            my_id = e;
            my_key = m;
        }
        if ((e & 31) == lane) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (lane + 32 * i == e)
                    key[i] = 0u;
            refresh();
        }
    }

    float w = 0.f;
    const bool chosen = lane < a.k && my_key > kKeyMasked;
    const float xj = chosen ? load_logit(row + my_id) : -INFINITY;
    if (a.renorm) {
        // all k scores times exp(-m), m the largest chosen logit (sigmoid: or 0):
        // the ratios are the same, and they survive where every score underflows
        float m = warp_max(xj);
        if (sigmoid)
            m = fminf(m, 0.f);
        if (chosen)
            w = sigmoid ? 1.0f / (expf(m) + expf(m - xj)) : expf(xj - m);
        const float total = warp_sum(w);
        w = chosen ? w / total : 0.f;
    } else if (chosen) {
        w = sigmoid ? sigmoid_f32(xj) : expf(xj - top) / sum;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = my_id;
        a.w[t * a.k + lane] = w * a.scale;
    }
}

template <typename TL, int NI>
__global__ void __launch_bounds__(256) moe_route_kernel(MoeRouteArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ float route_vals[];  // [warps][E] with groups
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * nw + warp; t < a.T;
         t += static_cast<int64_t>(gridDim.x) * nw)
        route_token<TL, NI>(a, t, lane, route_vals + warp * a.E);
}

template <typename TL>
cudaError_t launch_route_type(const MoeRouteArgs& a, int grid, int warps, cudaStream_t s)
{
    const size_t smem = a.n_group > 1 ? sizeof(float) * a.E * warps : 0;
    if (a.E <= 128)
        return launch_pdl(moe_route_kernel<TL, 4>, grid, 32 * warps, smem, s, a);
    if (a.E <= 256)
        return launch_pdl(moe_route_kernel<TL, 8>, grid, 32 * warps, smem, s, a);
    if (a.E <= 384)
        return launch_pdl(moe_route_kernel<TL, 12>, grid, 32 * warps, smem, s, a);
    if (a.E <= 512)
        return launch_pdl(moe_route_kernel<TL, 16>, grid, 32 * warps, smem, s, a);
    return launch_pdl(moe_route_kernel<TL, 32>, grid, 32 * warps, smem, s, a);
}

// Gradient of the weights at the logits, one warp per token.  With g = dL/dw
// and w the weights the router returned (0 in a slot that nothing could fill):
//   sigmoid  dx_i = w_i (1 - s_i) (g_i - r)      softmax, renormalised  dx_i = w_i (g_i - r)
//   softmax  dx_i = [i chosen] w_i g_i - p_i sum_j g_j w_j
// where r = sum_j g_j w_j / scale when renormalised, else 0.  All but the last
// are zero outside the chosen experts.  The row is put together in shared
// memory and written once.
template <typename TL>
__global__ void __launch_bounds__(256) moe_route_backward_kernel(MoeRouteBwdArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ float bwd_rows[];  // [warps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float* out = bwd_rows + warp * a.E;
    const bool sigmoid = a.scoring == CHORD_SCORE_SIGMOID;
    const bool dense = !sigmoid && !a.renorm;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * nw + warp; t < a.T;
         t += static_cast<int64_t>(gridDim.x) * nw) {
        const TL* row = static_cast<const TL*>(a.logits) + t * a.ld;
        int id = -1;
        float g = 0.f, w = 0.f;
        if (lane < a.k) {
            id = a.ids[t * a.k + lane];
            g = a.d_w[t * a.k + lane];
            w = a.w[t * a.k + lane];
            if (id < 0 || id >= a.E) {
                id = -1;  // (no such expert: no gradient)
                w = 0.f;
            }
        }
        const float gw = w != 0.f ? g * w : 0.f;
        const float dot = warp_sum(gw);
        float v = gw;
        if (a.renorm)
            v = w != 0.f ? w * (g - dot / a.scale) : 0.f;
        if (sigmoid && w != 0.f)
            v *= 1.0f / (1.0f + expf(load_logit(row + id)));  // 1 - s
        if (dense) {
            float top = -INFINITY;
            for (int e = lane; e < a.E; e += 32) {
                const float x = load_logit(row + e);
                out[e] = x;
                top = fmaxf(top, x);
            }
            top = warp_max(top);
            if (top == -INFINITY)
                top = 0.f;
            float sum = 0.f;
            for (int e = lane; e < a.E; e += 32) {
                const float p = expf(out[e] - top);
                out[e] = p;
                sum += p;
            }
            sum = warp_sum(sum);
            const float f = sum > 0.f ? -dot / sum : 0.f;
            for (int e = lane; e < a.E; e += 32)
                out[e] *= f;
        } else {
            for (int e = lane; e < a.E; e += 32)
                out[e] = 0.f;
        }
        __syncwarp();
        if (id >= 0)
            atomicAdd(out + id, v);
        __syncwarp();
        TL* dst = static_cast<TL*>(a.d_logits) + t * a.E;
        for (int e = lane; e < a.E; e += 32)
            dst[e] = from_f32<TL>(out[e]);
        __syncwarp();
    }
}

// Blocks of one warp spread a small batch over the SMs; larger ones take 8.
int warps_per_block(int64_t T, int sms) { return T <= 8 * static_cast<int64_t>(sms) ? 1 : 8; }

int blocks_for(int64_t T, int warps)
{
    const int64_t b = (T + warps - 1) / warps;
    return static_cast<int>(b < 65535 ? b : 65535);
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, int sms, cudaStream_t s)
{
    const int warps = warps_per_block(a.T, sms), grid = blocks_for(a.T, warps);
    return with_type(a.type, [&](auto v) { return launch_route_type<decltype(v)>(a, grid, warps, s); });
}

cudaError_t launch_moe_route_backward(const MoeRouteBwdArgs& a, int sms, cudaStream_t s)
{
    const int warps = warps_per_block(a.T, sms), grid = blocks_for(a.T, warps);
    const size_t smem = sizeof(float) * a.E * warps;
    return with_type(a.type, [&](auto v) {
        return launch_pdl(moe_route_backward_kernel<decltype(v)>, grid, 32 * warps, smem, s, a);
    });
}

}  // namespace chord
