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
// A token takes 16 lanes (up to 256 experts and 16 choices; a wave so has four) or
// a wave, each lane V experts.  A logit and its expert are one number whose order is
// the choice's: the bits of the logit as an integer in its order, then the expert,
// the lowest on top.  For bf16 logits that is a 32-bit integer; for binary32 ones 42
// bits, held exactly in a binary64 number, whose maximum is one instruction as well.
// Each lane sorts its V of them by a network of maxima and minima; a choice then
// is one maximum over the lanes (DPP), and the lane that held it moves up its next
// one.  No ties are left to look for.  (With a wave a token, a ballot for the lane
// that holds the maximum and its other experts looked through again for each choice,
// 16384 tokens of 256 experts, 8 choices took 15.0 us, of 64, 6 choices 8.8; now 8.4
// and 4.5 with the logits in a cache, 10.0 and 4.9 without; back 12.6 and 6.5, now 7.6
// and 3.8, 9.8 and 4.2 without.)  Forward bound by the vector instructions: 1007 a wave
// of four tokens, whose 4 cycles each are 82 % of the compute units' busy ones (of 1024
// experts 1317 a wave, 84 %); backward, 419, by the bytes.
#include "exp_device.hpp"
#include "fp4_device.hpp"
#include "fp4_launch.hpp"
#include "wave.hpp"

namespace fp4dev {
namespace {

constexpr int kOut = (int)0x807FFFFF;                  // -infinity

// An integer in the order of the binary32 values, one for both zeros; NaN as -infinity.
__device__ __forceinline__ int order_key(float v) {
    const int b = __float_as_int(v + 0.0f);
    return v != v ? kOut : b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float key_value(int key) {
    return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF));
}

constexpr int kExpertBits = 10;
constexpr int kLastExpert = (1 << kExpertBits) - 1;

// A logit with its expert; 0 for what is no choice, positive else.
template <bool BF16>
struct Pair;

template <>
struct Pair<true> {
    int v;
    static __device__ __forceinline__ Pair none() { return {0}; }
    // a bf16 value's key has its low 16 bits all alike
    static __device__ __forceinline__ Pair of(int key, int e) {
        const int p = (int)(((uint32_t)key ^ 0x80000000u) >> 16 << kExpertBits) | (kLastExpert - e);
        return {key > kOut ? p : 0};
    }
    __device__ __forceinline__ int expert() const { return kLastExpert - (v & kLastExpert); }
    __device__ __forceinline__ float logit() const {
        const int k = (int)((uint32_t)(v >> kExpertBits) << 16 ^ 0x80000000u);
        return key_value(k < 0 ? k | 0xFFFF : k);
    }
    static __device__ __forceinline__ Pair larger(Pair a, Pair b) { return {max(a.v, b.v)}; }
    static __device__ __forceinline__ Pair smaller(Pair a, Pair b) { return {min(a.v, b.v)}; }
    template <int CTRL>
    __device__ __forceinline__ Pair from() const { return {moved<CTRL, 0xF>(v, v)}; }
    __device__ __forceinline__ Pair of_lane(int lane) const { return {__builtin_amdgcn_readlane(v, lane)}; }
    __device__ __forceinline__ bool same(Pair o) const { return v == o.v; }
    __device__ __forceinline__ bool any() const { return v != 0; }
};

template <>
struct Pair<false> {
    double v;
    static __device__ __forceinline__ Pair none() { return {0.0}; }
    static __device__ __forceinline__ Pair of(int key, int e) {
        const bool in = key > kOut;
        const uint32_t bits = in ? (uint32_t)key ^ 0x80000000u : 0, last = in ? kLastExpert - e : 0;
        return {__builtin_fma((double)bits, 1024.0, (double)last)};
    }
    __device__ __forceinline__ uint32_t bits() const { return (uint32_t)(v * 0x1p-10); }      // truncated
    __device__ __forceinline__ int expert() const {
        return kLastExpert - (int)__builtin_fma((double)bits(), -1024.0, v);
    }
    __device__ __forceinline__ float logit() const { return key_value((int)(bits() ^ 0x80000000u)); }
    static __device__ __forceinline__ Pair larger(Pair a, Pair b) { return {__builtin_fmax(a.v, b.v)}; }
    static __device__ __forceinline__ Pair smaller(Pair a, Pair b) { return {__builtin_fmin(a.v, b.v)}; }
    template <int CTRL>
    __device__ __forceinline__ Pair from() const {
        const int lo = __double2loint(v), hi = __double2hiint(v);
        return {__hiloint2double(moved<CTRL, 0xF>(hi, hi), moved<CTRL, 0xF>(lo, lo))};
    }
    __device__ __forceinline__ Pair of_lane(int lane) const {
        return {__hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                                 __builtin_amdgcn_readlane(__double2loint(v), lane))};
    }
    __device__ __forceinline__ bool same(Pair o) const { return v == o.v; }
    __device__ __forceinline__ bool any() const { return v != 0.0; }
};

// The largest of a token's lanes, in all of them.
template <int LANES, typename P>
__device__ __forceinline__ P largest(P p) {
    p = P::larger(p, p.template from<kRowRor1>());
    p = P::larger(p, p.template from<kRowRor2>());
    p = P::larger(p, p.template from<kRowRor4>());
    p = P::larger(p, p.template from<kRowRor8>());
    if constexpr (LANES == 64) {
        p = P::larger(p, p.template from<kRowBcast15>());
        p = P::larger(p, p.template from<kRowBcast31>());
        p = p.of_lane(63);
    }
    return p;
}

template <int LANES>
__device__ __forceinline__ float token_sum(float v) {
    if constexpr (LANES == 64) return wave_sum(v);
    else return row_sum(v);
}

// Descending, by Batcher's odd-even merges.
template <int V, typename P>
__device__ __forceinline__ void sort_lane(P* p) {
#pragma unroll
    for (int run = 1; run < V; run <<= 1)
#pragma unroll
        for (int step = run; step >= 1; step >>= 1)
#pragma unroll
            for (int j = step % run; j + step < V; j += 2 * step)
#pragma unroll
                for (int i = 0; i < step; ++i) {
                    const int a = i + j, b = i + j + step;
                    if (b < V && a / (2 * run) == b / (2 * run)) {
                        const P hi = P::larger(p[a], p[b]), lo = P::smaller(p[a], p[b]);
                        p[a] = hi;
                        p[b] = lo;
                    }
                }
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (BF16) return bf16_value(static_cast<const uint16_t*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}

// exp(l - top), 1 where they are equal (also infinite); l <= top
__device__ __forceinline__ float score_over(float l, float top) {
    const float s = exp_minus(top - l);
    return l == top ? 1.0f : s;
}

// -log(1 + exp(-l)); what the logarithm loses next to 1 is a rounding of an exponent
__device__ __forceinline__ float log_sigmoid(float l) {
    return fminf(l, 0.0f) - 0.693147181f * __builtin_amdgcn_logf(1.0f + exp_minus(fabsf(l)));
}

// sigma and sigma (1 - sigma), without a difference of near values
__device__ __forceinline__ void sigmoid_and_slope(float l, float* s, float* slope) {
    const float e = exp_minus(fabsf(l)), r = __builtin_amdgcn_rcpf(1.0f + e);
    *s = l < 0.0f ? e * r : r;
    *slope = e * r * r;
}

// Expert i of a lane's V: four neighbours each, so that 16 lanes load whole lines.
template <int LANES, int V>
__device__ __forceinline__ int expert_at(int i) {
    constexpr int kRun = V < 4 ? V : 4;
    return (LANES * (i / kRun) + (threadIdx.x & (LANES - 1))) * kRun + i % kRun;
}

// The logits of a lane's experts, -infinity past the last one; `whole`: rows of E % 4
// == 0 elements at aligned addresses, four in one load (16384 x 256, softmax over all:
// fp32 10.1 us and 10.5 one by one, bf16 7.3 and 10.6; back 10.7 and 15.4, 8.0 and 12.9).
template <int LANES, int V, bool BF16>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, bool whole, float* l) {
    if (V >= 4 && whole) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int e = expert_at<LANES, V>(i);
            if constexpr (BF16) {
                const uint2 q = e < E ? *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + t * E + e)
                                      : make_uint2(0xFF80FF80u, 0xFF80FF80u);
                l[i] = bf16_lo(q.x), l[i + 1] = bf16_hi(q.x), l[i + 2] = bf16_lo(q.y), l[i + 3] = bf16_hi(q.y);
            } else {
                const float4 q = e < E ? *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + t * E + e)
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                l[i] = q.x, l[i + 1] = q.y, l[i + 2] = q.z, l[i + 3] = q.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_at<LANES, V>(i);
            l[i] = e < E ? load_logit<BF16>(logits, t * E + e) : -INFINITY;
        }
    }
}

// The scores of a lane's logits over the largest one, 0 for what is no choice, and
// their sum over the token's lanes: the forward pass divides by it and the backward
// pass by the same bits.  Equal logits err the same way, so the exponential is one
// whose error does not grow with its argument: hundreds of them would leave it whole
// in the sum.
template <int LANES, int V>
__device__ __forceinline__ float scores(const float* l, float top, float* s) {
#pragma unroll
    for (int i = 0; i < V; ++i)                        // of a NaN and 200 the minimum is 200
        s[i] = exp_minus_to_200(fminf(top - l[i], 200.0f));
    if (__any(top == INFINITY)) {                      // no number to subtract; other tokens' stay as they are
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = l[i] == INFINITY ? 1.0f : s[i];
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += s[i];
    return token_sum<LANES>(sum);
}

// A workgroup is a wave: its tokens' first one, and this lane's.
template <int LANES>
__device__ __forceinline__ int64_t token_of() {
    return (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * (64 / LANES) + threadIdx.x / LANES;
}

// K: the most choices, of which no lane holds more.
template <int LANES, int V, int K, bool BF16>
__global__ __launch_bounds__(64) void moe_route(const void* __restrict__ logits, int64_t tokens, int E, bool whole, int k,
                                                bool sigmoid, bool normalize, int* __restrict__ ids,
                                                float* __restrict__ weights) {
    constexpr int kKept = V < K ? V : K;
    using P = Pair<BF16>;
    const int64_t mine = token_of<LANES>(), t = mine < tokens ? mine : tokens - 1;
    const int lane = threadIdx.x & (LANES - 1);
    float l[V];
    load_logits<LANES, V, BF16>(logits, t, E, whole, l);
    P p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = P::of(order_key(l[i]), expert_at<LANES, V>(i));
    sort_lane<V>(p);
    P m = largest<LANES>(p[0]), chosen = P::none();
    const float top = m.logit();
    float total = 1.0f;
    if (!sigmoid && !normalize) {
        float s[V];
        total = scores<LANES, V>(l, top, s);
    }
    for (int j = 0;;) {
        if (lane == j) chosen = m;
        if (++j == k) break;
        if (p[0].same(m)) {                            // nothing left: all lanes, and none again
#pragma unroll
            for (int i = 0; i + 1 < kKept; ++i) p[i] = p[i + 1];
            p[kKept - 1] = P::none();
        }
        m = largest<LANES>(p[0]);
    }
    const float c = chosen.logit();
    float w = 0.0f, slope;
    if (!sigmoid) w = score_over(c, top);
    else if (normalize) w = score_over(log_sigmoid(c), log_sigmoid(top));
    else sigmoid_and_slope(c, &w, &slope);
    if (!chosen.any()) w = 0.0f;
    if (normalize) total = token_sum<LANES>(w);
    if (lane < k && mine < tokens) {
        ids[t * k + lane] = chosen.any() ? chosen.expert() : -1;
        weights[t * k + lane] = chosen.any() ? w * __builtin_amdgcn_rcpf(total) : 0.0f;
    }
}

template <int LANES, int V, bool BF16>
__global__ __launch_bounds__(64) void moe_route_back(const float* __restrict__ dweights,
                                                     const void* __restrict__ logits, const int* __restrict__ ids,
                                                     int64_t tokens, int E, bool whole, int k, bool sigmoid,
                                                     bool normalize, void* __restrict__ dlogits) {
    // by token and expert: its gradient, or that of its weight
    __shared__ __attribute__((aligned(16))) float row[64 * V];
    const int64_t mine = token_of<LANES>(), t = mine < tokens ? mine : tokens - 1;
    const int lane = threadIdx.x & (LANES - 1);
    float* const at = row + threadIdx.x / LANES * (LANES * V);
    const bool dense = !sigmoid && !normalize;
    float l[V], s[V];
    if (dense) load_logits<LANES, V, BF16>(logits, t, E, whole, l);
    const int id = lane < k ? ids[t * k + lane] : -1;
    const float given = lane < k ? dweights[t * k + lane] : 0.0f;
    const float c = id >= 0 && id < E ? load_logit<BF16>(logits, t * E + id) : -INFINITY;
    const bool chosen = c > -INFINITY;                 // not for a NaN
    const float g = chosen ? given : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) at[expert_at<LANES, V>(i)] = 0.0f;
    float inner = 0.0f, d = g, r = 1.0f;
    if (dense) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);                // a NaN is none
        m = token_max<LANES>(m);
        const float total = scores<LANES, V>(l, m, s);
        r = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;        // where nothing is a choice
        inner = token_sum<LANES>(chosen ? g * (score_over(c, m) * r) : 0.0f);
    } else {
        float sigma = 0.0f, slope = 0.0f, w = 0.0f;
        sigmoid_and_slope(c, &sigma, &slope);
        if (normalize) {
            const float top = token_max<LANES>(chosen ? c : -INFINITY);
            if (chosen) w = sigmoid ? score_over(log_sigmoid(c), log_sigmoid(top)) : score_over(c, top);
            w *= __builtin_amdgcn_rcpf(token_sum<LANES>(w));
            inner = token_sum<LANES>(chosen ? g * w : 0.0f);
            d = w * (g - inner);
            // 1 - sigma(c) = sigma(-c)
            if (sigmoid) sigmoid_and_slope(-c, &sigma, &slope), d *= sigma;
        } else {
            d = g * slope;
        }
    }
    __syncthreads();                                   // of one wave: the row's values are in place
    if (chosen) at[id] = d;
    __syncthreads();
    if (mine >= tokens) return;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = at[expert_at<LANES, V>(i)];
        // zero for what is no choice, also where a gradient of the weights is no number
        if (dense) v[i] = s[i] != 0.0f ? s[i] * r * (v[i] - inner) : 0.0f;
    }
    if (V >= 4 && whole) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int e = expert_at<LANES, V>(i);
            if (e >= E) continue;
            if constexpr (BF16)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dlogits) + t * E + e) =
                    make_uint2(bf16_pair(v[i], v[i + 1]), bf16_pair(v[i + 2], v[i + 3]));
            else
                *reinterpret_cast<float4*>(static_cast<float*>(dlogits) + t * E + e) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_at<LANES, V>(i);
            if (e >= E) continue;
            if constexpr (BF16) static_cast<uint16_t*>(dlogits)[t * E + e] = (uint16_t)bf16_rne(v[i]);
            else static_cast<float*>(dlogits)[t * E + e] = v[i];
        }
    }
}

template <int LANES, int V, int K>
hipError_t launch_v(const float* dweights, const void* logits, int bf16, int64_t tokens, int64_t E, int64_t k,
                    int sigmoid, int normalize, int* ids, float* weights, void* dlogits, hipStream_t st) {
    const dim3 grid = grid_of((tokens + 64 / LANES - 1) / (64 / LANES), 64), block(64);
    const uintptr_t to = bf16 ? 8 : 16;
    const bool whole = E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % to == 0 &&
                       reinterpret_cast<uintptr_t>(dlogits) % to == 0;
    if (dlogits) {
        auto* const back = bf16 ? &moe_route_back<LANES, V, true> : &moe_route_back<LANES, V, false>;
        return launch(back, grid, block, st, dweights, logits, (const int*)ids, tokens, (int)E, whole, (int)k,
                      sigmoid != 0, normalize != 0, dlogits);
    }
    auto* const route = bf16 ? &moe_route<LANES, V, K, true> : &moe_route<LANES, V, K, false>;
    return launch(route, grid, block, st, logits, tokens, (int)E, whole, (int)k, sigmoid != 0, normalize != 0, ids,
                  weights);
}

hipError_t launch_any(const float* dweights, const void* logits, int bf16, int64_t tokens, int64_t E, int64_t k,
                      int sigmoid, int normalize, int* ids, float* weights, void* dlogits, hipStream_t st) {
    // a wave a token takes what 16 lanes cannot, which is slower wherever they can (the
    // comment at the top); of the 16 that a lane sorts it keeps no more than can be
    // chosen from it (16384 x 256, 8 choices, softmax over all: 9.8 us with 8 kept,
    // 12.2 with 16)
    auto* run = E <= 64 ? &launch_v<64, 1, 64> : E <= 128 ? &launch_v<64, 2, 64> : E <= 256 ? &launch_v<64, 4, 64>
                : E <= 512 ? &launch_v<64, 8, 64> : &launch_v<64, 16, 64>;
    if (k <= 16 && E <= 256)
        run = E <= 16 ? &launch_v<16, 1, 16> : E <= 32 ? &launch_v<16, 2, 16> : E <= 64 ? &launch_v<16, 4, 16>
              : E <= 128 ? &launch_v<16, 8, 16> : k <= 8 ? &launch_v<16, 16, 8> : &launch_v<16, 16, 16>;
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
