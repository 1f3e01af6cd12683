// Routing of tokens to experts: per token row of logits [E], scores (softmax
// or sigmoid), an optional balance bias that only the choice sees, optional
// expert groups of which the best few are kept, the top_k experts in order of
// choice, and their weights.
//
//   score  s = exp(l - max l) / sum exp(l - max l)   or   1 / (1 + exp(-l))
//   pick     = l without a bias (both scores rise with l, so the order is the
//              same and no rounding of the score can make a tie), s + bias with
//   a group's rank = its best pick, or with a bias the sum of its two best
//   ids    = the top_k picks among the kept groups, equal picks in order of
//            index;  w = s at the ids [/ their sum] * scale
// A logit of -inf or NaN takes the expert out for the token; a slot that no
// expert is left for gets id -1 and weight 0.
//
// One wave per token: lane l holds experts l, l + 64, ...  A round of the
// choice is a wave maximum of order-preserving integer keys; the lowest index
// among equals falls out of the ballot of (key == maximum), expert row by
// expert row.
#include "common.h"

namespace llmint8 {

namespace {

// float -> unsigned key of the same order; finite values and infinities map
// above 0, which is kept for "not available".  -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __builtin_bit_cast(float, k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

template <int DT>  // LLMINT8_F16, LLMINT8_BF16, LLMINT8_F32
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (DT == LLMINT8_F32)
        return static_cast<const float*>(p)[i];
    else
        return widen16<DT == LLMINT8_BF16>(static_cast<const uint16_t*>(p)[i]);
}

constexpr int kRouteWaves = 4;

// One token; keys: this wave's E words of LDS (used with groups only).
template <int DT, int V>  // V: experts per lane, E <= 64 V
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int lane, uint32_t* keys) {
    float l[V];
    bool alive[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 64 * v + lane;
        l[v] = e < a.E ? load_logit<DT>(a.logits, t * a.E + e) : -__builtin_inff();
        alive[v] = l[v] > -__builtin_inff();  // false for NaN
    }
    // scores; softmax's are left unnormalized (total holds their sum)
    float s[V], total = 1.0f;
    if (a.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = 1.0f / (1.0f + expf(-l[v]));
    } else {
        float top = -__builtin_inff();
#pragma unroll
        for (int v = 0; v < V; ++v) top = alive[v] ? fmaxf(top, l[v]) : top;
        top = wave_max(top);
        total = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {  // (l == top: also for an infinite maximum)
            s[v] = alive[v] ? (l[v] == top ? 1.0f : expf(l[v] - top)) : 0.0f;
            total += s[v];
        }
        total = wave_add(total);
    }
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 64 * v + lane;
        float p = l[v];
        if (a.bias != nullptr && e < a.E) p = (a.sigmoid ? s[v] : s[v] / total) + a.bias[e];
        key[v] = alive[v] && p > -__builtin_inff() ? order_key(p) : 0u;
    }
    if (a.n_group > 1) {
        wave_fence();  // the last token's reads
        // group g's keys are read by the P lanes g P .. g P + P - 1
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (64 * v + lane < a.E) keys[64 * v + lane] = key[v];
        wave_fence();
        const int size = a.E / a.n_group;
        const int P = a.group_lanes, g = lane / P;
        uint32_t best = 0, next = 0;
        if (g < a.n_group)
            for (int j = lane - g * P; j < size; j += P) {
                const uint32_t k = keys[g * size + j];
                next = max(next, min(best, k));
                best = max(best, k);
            }
        for (int m = 1; m < P; m <<= 1) {
            const uint32_t b = __shfl_xor(best, m), n = __shfl_xor(next, m);
            next = max(max(next, n), min(best, b));
            best = max(best, b);
        }
        uint32_t rank = best;
        if (a.bias != nullptr && next != 0) {
            const float two = key_value(best) + key_value(next);
            rank = two == two ? order_key(two) : 0u;
        }
        // groups ranked above this lane's, the lower index first among equals
        int above = 0;
        for (int o = 0; o < a.n_group; ++o) {
            const uint32_t r = (uint32_t)__builtin_amdgcn_readlane((int)rank, o * P);
            above += r > rank || (r == rank && o < g);
        }
        const uint64_t kept = __ballot(g < a.n_group && above < a.topk_group);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = 64 * v + lane;
            const int eg = e < a.E ? e / size : 0;
            if (!((kept >> (eg * P)) & 1)) key[v] = 0;
        }
    }
    // top_k rounds; lane j keeps slot j
    int my_id = -1;
    float my_s = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = max(m, key[v]);
        m = wave_max_u32(m);
        if (m == 0) break;  // (uniform) no expert is left
        int id = -1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint64_t hit = __ballot(key[v] == m);
            if (id < 0 && hit != 0) {
                const int at = __builtin_ctzll(hit);
                id = 64 * v + at;
                const float sv = __builtin_bit_cast(
                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s[v]), at));
                if (lane == at) key[v] = 0;
                if (lane == j) {
                    my_id = id;
                    my_s = sv;
                }
            }
        }
    }
    float w = my_s;
    if (a.renormalize) {
        const float sum = wave_add(lane < a.top_k ? my_s : 0.0f);
        w = sum > 0.0f ? my_s / sum : 0.0f;
    } else if (!a.sigmoid) {
        w = my_id >= 0 ? my_s / total : 0.0f;
    }
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = my_id;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

template <int DT, int V>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
    extern __shared__ uint32_t keys_all[];  // groups only: E keys per wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // (waves run on their own: no workgroup barrier below)
    for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < a.T; t += (int64_t)gridDim.x * kRouteWaves)
        route_token<DT, V>(a, t, lane, keys_all + wave * a.E);
}

template <int DT>
hipError_t launch_route_dt(const RouteArgs& a, hipStream_t stream) {
    const int64_t want = (a.T + kRouteWaves - 1) / kRouteWaves;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536)), block(64 * kRouteWaves);
    const size_t lds = a.n_group > 1 ? (size_t)kRouteWaves * a.E * 4 : 0;
    if (a.E <= 64)
        route_kernel<DT, 1><<<grid, block, lds, stream>>>(a);
    else if (a.E <= 128)
        route_kernel<DT, 2><<<grid, block, lds, stream>>>(a);
    else if (a.E <= 256)
        route_kernel<DT, 4><<<grid, block, lds, stream>>>(a);
    else if (a.E <= 512)
        route_kernel<DT, 8><<<grid, block, lds, stream>>>(a);
    else
        route_kernel<DT, 16><<<grid, block, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& in, int dtype, hipStream_t stream) {
    RouteArgs a = in;
    int pow2 = 1;
    while (pow2 < a.n_group) pow2 <<= 1;
    a.group_lanes = 64 / pow2;
    if (dtype == LLMINT8_F32) return launch_route_dt<LLMINT8_F32>(a, stream);
    if (dtype == LLMINT8_BF16) return launch_route_dt<LLMINT8_BF16>(a, stream);
    return launch_route_dt<LLMINT8_F16>(a, stream);
}

}  // namespace llmint8
