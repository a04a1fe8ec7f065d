// moe_route.hip -- the router of a mixture of experts: each token's k best
// experts and their weights, and the gradient of the weights.
//
// l: a token's logits; chosen: its k largest, largest first, equal ones by
// their index.  Scores a_i and weights w_j of the chosen:
//     softmax   a_i = exp(l_i - m), m = max l     w_j = a_j / sum a  (over all, or the chosen)
//     sigmoid   a_i = 1 / (1 + exp(-l_i))         w_j = a_j, or a_j / sum a over the chosen
// The choice goes by the logits themselves, of which both scores are increasing
// functions: no rounding of a score decides.  The sigmoid's normalized weights
// go by way of log a, whose differences stay where all scores of a token leave
// binary32 (logits below -104).  An infinite largest logit counts as
// exp(0) against itself and exp(-inf) against the rest.  -infinity and NaN are
// no choice: id -1, weight 0 where nothing else is left.
//
// Backward, g the gradient of w (0 where not chosen), c = sum_j g_j w_j:
//     softmax              dl_i = p_i (g_i - c), p = a / sum a, over all experts
//     softmax, normalized  dl_j = w_j (g_j - c)
//     sigmoid              dl_j = g_j a_j (1 - a_j)
//     sigmoid, normalized  dl_j = (1 - a_j) w_j (g_j - c)
//
// A wave takes a token.  A choice is one maximum over the wave (DPP, wave.hpp) of
// order-preserving integers, then a ballot for the lane that holds it; only where
// several hold the same value is the lowest index looked for.
#include "fp4_device.hpp"
#include "fp4_launch.hpp"
#include "wave.hpp"

namespace fp4dev {
namespace {

constexpr int kWaves = 4;
constexpr int kNothing = INT32_MIN;                    // past the experts, or chosen already
constexpr int kOut = (int)0x807FFFFF;                  // -infinity

// An integer in the order of the binary32 values, one for both zeros; NaN as -infinity.
__device__ __forceinline__ int order_key(float v) {
    const int b = __float_as_int(v + 0.0f);
    return v != v ? kOut : b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float key_value(int key) {
    return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF));
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (BF16) return bf16_value(static_cast<const uint16_t*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}

// exp(l - top), 1 where they are equal (also infinite); l <= top
__device__ __forceinline__ float score_over(float l, float top) { return l == top ? 1.0f : expf(l - top); }

__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }

// sigma and sigma (1 - sigma), without a difference of near values
__device__ __forceinline__ void sigmoid_and_slope(float l, float* s, float* slope) {
    const float e = expf(-fabsf(l)), r = 1.0f / (1.0f + e);
    *s = l < 0.0f ? e * r : r;
    *slope = e * r * r;
}

// The keys of a token's logits, element i of lane's at expert 64 i + lane.
template <int V, bool BF16>
__device__ __forceinline__ void load_keys(const void* logits, int64_t t, int E, int lane, int* key) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        key[i] = e < E ? order_key(load_logit<BF16>(logits, t * E + e)) : kNothing;
    }
}

// sum over the token's experts of exp(l - top)
template <int V>
__device__ __forceinline__ float sum_scores(const int* key, float top) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (key[i] > kOut) s += score_over(key_value(key[i]), top);
    return wave_sum(s);
}

// a wave's token, the last one again where there is none (its results are not stored)
__device__ __forceinline__ int64_t token_of(int64_t tokens, bool* live) {
    const int64_t t = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * kWaves + wave_uniform(threadIdx.x >> 6);
    *live = t < tokens;
    return *live ? t : tokens - 1;
}

template <int V, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void moe_route(const void* __restrict__ logits, int64_t tokens, int E, int k,
                                                         bool sigmoid, bool normalize, int* __restrict__ ids,
                                                         float* __restrict__ weights) {
    bool live;
    const int64_t t = token_of(tokens, &live);
    if (!live) return;
    const int lane = threadIdx.x & 63;
    int key[V];
    load_keys<V, BF16>(logits, t, E, lane, key);
    // the lane's largest key and the first of its elements that has it
    int best = kNothing, at = 0;
    auto look = [&] {
        best = key[V - 1];
        at = V - 1;
#pragma unroll
        for (int i = V - 2; i >= 0; --i) {
            at = key[i] >= best ? i : at;
            best = max(best, key[i]);
        }
    };
    look();
    int m = wave_max(best), id = -1;
    const float top = key_value(m);
    float total = 1.0f, l = 0.0f;
    if (!sigmoid && !normalize) total = sum_scores<V>(key, top);
    for (int j = 0; j < k && m > kOut; ++j) {          // the same for the whole wave
        const uint64_t holders = __ballot(best == m);
        int chosen;
        if (holders & (holders - 1)) {
            chosen = wave_min(best == m ? 64 * at + lane : INT32_MAX);
        } else {
            const int holder = __builtin_ctzll(holders);
            chosen = 64 * __builtin_amdgcn_readlane(at, holder) + holder;
        }
        if (lane == j) {
            id = chosen;
            l = key_value(m);
        }
        if (lane == (chosen & 63)) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = i == at ? kNothing : key[i];
            look();
        }
        m = wave_max(best);
    }
    float w = 0.0f;
    if (sigmoid) {
        float slope;
        if (normalize) w = score_over(log_sigmoid(l), log_sigmoid(top));
        else sigmoid_and_slope(l, &w, &slope);
    } else {
        w = score_over(l, top);
    }
    if (id < 0) w = 0.0f;
    if (normalize) total = wave_sum(w);
    if (lane < k) {
        ids[t * k + lane] = id;
        weights[t * k + lane] = id < 0 ? 0.0f : w / total;
    }
}

template <int V, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void moe_route_back(const float* __restrict__ dweights,
                                                              const void* __restrict__ logits,
                                                              const int* __restrict__ ids, int64_t tokens, int E, int k,
                                                              bool sigmoid, bool normalize, void* __restrict__ dlogits) {
    __shared__ float row[kWaves][64 * V];              // by expert: its gradient, or that of its weight
    bool live;
    const int64_t t = token_of(tokens, &live);
    const int lane = threadIdx.x & 63;
    float* const mine = row[threadIdx.x >> 6];
    int id = lane < k ? ids[t * k + lane] : -1;
    float g = lane < k ? dweights[t * k + lane] : 0.0f;
    int key = id >= 0 && id < E ? order_key(load_logit<BF16>(logits, t * E + id)) : kNothing;
    const bool chosen = key > kOut;
    if (!chosen) g = 0.0f;
    const float l = key_value(key);
#pragma unroll
    for (int i = 0; i < V; ++i) mine[64 * i + lane] = 0.0f;
    const bool dense = !sigmoid && !normalize;
    int every[V];
    float top = 0.0f, total = 1.0f, inner = 0.0f, d = g;
    if (dense) {
        load_keys<V, BF16>(logits, t, E, lane, every);
        int m = every[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = max(m, every[i]);
        top = key_value(wave_max(m));
        total = sum_scores<V>(every, top);
        inner = wave_sum(chosen ? g * (score_over(l, top) / total) : 0.0f);
    } else {
        float s = 0.0f, slope = 0.0f, w = 0.0f;
        if (sigmoid) sigmoid_and_slope(l, &s, &slope);
        if (normalize) {
            top = key_value(wave_max(key));
            if (chosen) w = sigmoid ? score_over(log_sigmoid(l), log_sigmoid(top)) : score_over(l, top);
            total = wave_sum(w);
            w = chosen ? w / total : 0.0f;
            inner = wave_sum(g * w);
            d = w * (g - inner);
            // 1 - sigma(l) = sigma(-l)
            if (sigmoid) sigmoid_and_slope(-l, &s, &slope), d *= s;
        } else {
            d = g * slope;
        }
    }
    __syncthreads();                                   // a wave's own row; every wave comes here
    if (chosen) mine[id] = d;
    __syncthreads();
    if (!live) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 64 * i + lane;
        if (e >= E) continue;
        float v = mine[e];
        if (dense) v = every[i] > kOut ? score_over(key_value(every[i]), top) / total * (v - inner) : 0.0f;
        if constexpr (BF16) static_cast<uint16_t*>(dlogits)[t * E + e] = (uint16_t)bf16_rne(v);
        else static_cast<float*>(dlogits)[t * E + e] = v;
    }
}

template <int V>
hipError_t launch_v(const float* dweights, const void* logits, int bf16, int64_t tokens, int64_t E, int64_t k,
                    int sigmoid, int normalize, int* ids, float* weights, void* dlogits, hipStream_t st) {
    const dim3 grid = grid_of((tokens + kWaves - 1) / kWaves, 64 * kWaves), block(64 * kWaves);
    if (dlogits) {
        auto* const back = bf16 ? &moe_route_back<V, true> : &moe_route_back<V, false>;
        return launch(back, grid, block, st, dweights, logits, (const int*)ids, tokens, (int)E, (int)k, sigmoid != 0,
                      normalize != 0, dlogits);
    }
    auto* const route = bf16 ? &moe_route<V, true> : &moe_route<V, false>;
    return launch(route, grid, block, st, logits, tokens, (int)E, (int)k, sigmoid != 0, normalize != 0, ids, weights);
}

hipError_t launch_any(const float* dweights, const void* logits, int bf16, int64_t tokens, int64_t E, int64_t k,
                      int sigmoid, int normalize, int* ids, float* weights, void* dlogits, hipStream_t st) {
    auto* const run = E <= 64 ? &launch_v<1> : E <= 128 ? &launch_v<2> : E <= 256 ? &launch_v<4>
                      : E <= 512 ? &launch_v<8> : &launch_v<16>;
    return run(dweights, logits, bf16, tokens, E, k, sigmoid, normalize, ids, weights, dlogits, st);
}

}  // namespace

hipError_t launch_moe_route(const void* logits, int bf16, int64_t tokens, int64_t experts, int64_t k, int sigmoid,
                            int normalize, int* ids, float* weights, hipStream_t st) {
    return launch_any(nullptr, logits, bf16, tokens, experts, k, sigmoid, normalize, ids, weights, nullptr, st);
}

hipError_t launch_moe_route_back(const float* dweights, const void* logits, int bf16, const int* ids, int64_t tokens,
                                 int64_t experts, int64_t k, int sigmoid, int normalize, void* dlogits, hipStream_t st) {
    return launch_any(dweights, logits, bf16, tokens, experts, k, sigmoid, normalize, const_cast<int*>(ids), nullptr,
                      dlogits, st);
}

}  // namespace fp4dev
