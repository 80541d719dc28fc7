// Routing to experts: the ids and gates of each token's experts from its logits, and the
// gradient of the gates.
//
//   s = softmax(l) or sigmoid(l);  key = s + bias, or l without one
//   expert groups: the top_groups of them with the largest key, or sum of two largest s + bias
//   ids = the fan largest keys in the open groups, in order, ties to the lowest index
//   gates = scale s[ids], or scale s[ids] / sum of s[ids]
//
// A row of 16 lanes takes a token (64 lanes past 256 experts), V logits a lane in registers;
// a reduction over a row is four rotations within it.  Each pick is one such reduction for
// the largest key and one for its lowest index.
//
// The selection is that of the formula in 64 bits.  Keys are computed in fp32 and the picks
// made with them; where two keys that decide (neighbours in the order, or the last one in and
// the first one out) are closer than their rounding errors, the wave makes its picks again
// from keys in 64 bits, some ten times slower and rare: so which experts a token gets does
// not hang on the order of a sum.  Without a bias the order is that of the logits and exact.
#include "route.h"

#include <algorithm>

#include "kernels.h"

namespace gemm_f16 {

// Waves of a workgroup: with expert groups a wave keeps its tokens' keys in LDS, 64 KB at most
// for all.
template <int L>
constexpr int kRouteWaves = L == 16 ? 4 : 2;

template <int CTRL>
__device__ __forceinline__ int rot(int x) {
    return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float rot(float x) {
    return __builtin_bit_cast(float, rot<CTRL>(__builtin_bit_cast(int, x)));
}
template <int CTRL>
__device__ __forceinline__ double rot(double x) {
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)rot<CTRL>((int)(uint32_t)v), hi = (uint32_t)rot<CTRL>((int)(uint32_t)(v >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// op over the L lanes of a token, the result in all of them.  The order of a sum is the same
// for every lane: lane i adds what lies opposite to it, and both orders of two terms agree.
template <int L, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T x, Op op) {
    x = op(x, rot<0x128>(x));  // rotations of a row by 8, 4, 2 and 1
    x = op(x, rot<0x124>(x));
    x = op(x, rot<0x122>(x));
    x = op(x, rot<0x121>(x));
    if constexpr (L == 64) {
        x = op(x, __shfl_xor(x, 16));
        x = op(x, __shfl_xor(x, 32));
    }
    return x;
}
template <int L, class T>
__device__ __forceinline__ T lanes_max(T x) {
    return lanes_reduce<L>(x, [](T a, T b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ int lanes_min(int x) {
    return lanes_reduce<L>(x, [](int a, int b) { return a < b ? a : b; });
}
template <int L, class T>
__device__ __forceinline__ T lanes_sum(T x) {
    return lanes_reduce<L>(x, [](T a, T b) { return a + b; });
}

// Expert of value v of a lane: blocks of up to 4 neighbours a lane; rising with v.
template <int L, int V>
struct Experts {
    static constexpr int B = V < 4 ? V : 4;
    static __device__ __forceinline__ int at(int v, int sub) { return v / B * (B * L) + sub * B + v % B; }
};

constexpr float kNone = -__builtin_inff();  // a key that is never picked

// The lane's logits; experts past the last, and NaN, as -inf.
template <int L, int V>
__device__ __forceinline__ void load_logits(const RouteParams &p, int64_t token, int sub, float (&l)[V]) {
    using E = Experts<L, V>;
#pragma unroll
    for (int v = 0; v < V; v += E::B) {
        const int e = E::at(v, sub);
        const int64_t at = token * p.experts + e;
        if (E::B == 4 && p.vec) {
            if (e < p.experts) {
                if (p.f32) {
                    const floatx4 x = *reinterpret_cast<const floatx4 *>(static_cast<const float *>(p.logits) + at);
#pragma unroll
                    for (int i = 0; i < E::B; ++i) l[v + i] = x[i];
                } else {
                    const half4 x = *reinterpret_cast<const half4 *>(static_cast<const _Float16 *>(p.logits) + at);
#pragma unroll
                    for (int i = 0; i < E::B; ++i) l[v + i] = (float)x[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < E::B; ++i) l[v + i] = kNone;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E::B; ++i)
                l[v + i] = e + i >= p.experts ? kNone
                           : p.f32            ? static_cast<const float *>(p.logits)[at + i]
                                              : (float)static_cast<const _Float16 *>(p.logits)[at + i];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = l[v] == l[v] ? l[v] : kNone;
}

__device__ __forceinline__ float load_logit(const RouteParams &p, int64_t token, int e) {
    const int64_t at = token * p.experts + e;
    return p.f32 ? static_cast<const float *>(p.logits)[at] : (float)static_cast<const _Float16 *>(p.logits)[at];
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// exp(l - m) for l <= m, 1 where they are the same infinity
template <class T>
__device__ __forceinline__ T exp_below(float l, float m) {
    return l == m ? T(1) : exp_of(T(l) - T(m));
}

template <class T>
__device__ __forceinline__ T sigmoid_of(float l) {
    return T(1) / (T(1) + exp_of(-T(l)));
}

// x of e / per for e below 2048: e + 1/2 is at least 1/4096 of per away from a border.
__device__ __forceinline__ int group_of(int e, float inv_per) { return (int)(((float)e + 0.5f) * inv_per); }

// exp(-m) sigmoid(l), m >= min(l, 0): sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)).  What
// renormalised gates are made of: the common factor keeps scores below fp32's range apart.
__device__ __forceinline__ float shifted_sigmoid(float l, float m) {
    return exp_below<float>(l < 0.0f ? l : 0.0f, m) / (1.0f + expf(-__builtin_fabsf(l)));
}

__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The experts of the wave's tokens: lane f % L of a token gets the f-th's id (-1: none left)
// in slot f / L.  lds: the wave's part, for the groups.  Returns whether the token's picks
// hang on differences below the keys' rounding errors (never for T = double).
template <class T, int L, int V>
__device__ __forceinline__ bool pick_experts(const RouteParams &p, const float (&l)[V], int sub, int row, char *lds,
                                             int (&id)[kRouteFan / 16]) {
    using E = Experts<L, V>;
    constexpr bool kExact = sizeof(T) == 8;
    T key[V], score[V];
    const bool by_score = p.bias != nullptr, need = by_score || (p.groups > 1 && p.group_top == 2);
    T largest = T(0);  // score, for the rounding errors
    if (need) {
        if (p.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) score[v] = sigmoid_of<T>(l[v]);
            largest = T(1);
        } else {
            float m = l[0];
#pragma unroll
            for (int v = 1; v < V; ++v) m = l[v] > m ? l[v] : m;
            m = lanes_max<L>(m);
            T sum = T(0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                score[v] = l[v] == kNone ? T(0) : exp_below<T>(l[v], m);
                sum += score[v];
            }
            sum = lanes_sum<L>(sum);
#pragma unroll
            for (int v = 0; v < V; ++v) score[v] /= sum;
            largest = T(1) / sum;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = E::at(v, sub);
        if (by_score) {
            const T k = score[v] + (e < p.experts ? T(p.bias[e]) : T(0));
            key[v] = l[v] == kNone || !(k == k) ? T(kNone) : k;
        } else {
            key[v] = T(l[v]);
        }
    }
    // What two keys can be off by against each other: a score by 2^-22 of itself (exp, a sum,
    // a quotient), a softmax's sum, which all scores share, by 2^-18 of itself, a key's last
    // rounding by 2^-24 of the key.  Twice that for sums of two.
    T error = T(0);
    if (!kExact && need) {
        T size = T(1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const T k = key[v] < T(0) ? -key[v] : key[v];
            size = by_score && k > size && k < T(__builtin_inff()) ? k : size;
        }
        error = lanes_max<L>(size) * T(0x1p-22) + (p.sigmoid ? T(0x1p-20) : largest * T(0x1p-17));
    }
    bool close = false;
    if (p.groups > 1) {
        // the group's largest key, or the sum of its two largest: lane g of a token takes
        // group g; a pad per group keeps the lanes on different banks
        const int per = p.experts / p.groups;
        const float inv_per = 1.0f / (float)per;
        T *const keys = reinterpret_cast<T *>(lds) + (int64_t)row * (p.experts + 2 * p.groups);
        T *const value = keys + p.experts + p.groups;
        wave_lds_fence();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = E::at(v, sub);
            if (e < p.experts) keys[e + group_of(e, inv_per)] = p.group_top == 2 && !by_score ? (l[v] == kNone ? T(kNone) : score[v]) : key[v];
        }
        wave_lds_fence();
        for (int g = sub; g < p.groups; g += L) {
            T first = T(kNone), second = T(kNone);
            const T *k = keys + g * (per + 1);
#pragma unroll 4
            for (int i = 0; i < per; ++i) {
                const T x = k[i], low = x < first ? x : first;
                first = x > first ? x : first;
                second = low > second ? low : second;
            }
            // (a group with one expert left counts that one alone)
            value[g] = p.group_top == 2 && second != T(kNone) ? first + second : first;
        }
        wave_lds_fence();
        uint64_t mine = 0;  // open groups, the bits of this lane's
        for (int g = sub; g < p.groups; g += L) {
            const T x = value[g];
            int rank = 0;
            for (int o = 0; o < p.groups; ++o) rank += value[o] > x || (value[o] == x && o < g);
            const bool open = rank < p.top_groups && x != T(kNone);
            mine |= (uint64_t)open << g;
            // the last one in, and another group within their errors
            if (!kExact && need && open && rank == p.top_groups - 1) {
                for (int o = 0; o < p.groups; ++o) {
                    const T y = value[o], d = x > y ? x - y : y - x;
                    if (o != g && d <= T(2) * error) close = true;
                }
            }
        }
        const uint32_t lo = (uint32_t)lanes_reduce<L>((int)(uint32_t)mine, [](int a, int b) { return a | b; });
        const uint32_t hi = (uint32_t)lanes_reduce<L>((int)(uint32_t)(mine >> 32), [](int a, int b) { return a | b; });
        const uint64_t open = (uint64_t)hi << 32 | lo;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = E::at(v, sub);
            if (e < p.experts && !((open >> group_of(e, inv_per)) & 1)) key[v] = T(kNone);
        }
    }
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) id[i] = -1;
    T before = T(0);
    // (one more than the picks: the first one out)
    const int turns = !kExact && by_score ? p.fan + 1 : p.fan;
    for (int f = 0; f < turns; ++f) {
        T m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
        m = lanes_max<L>(m);
        if (!kExact && by_score && f > 0 && m != T(kNone) && before - m <= error) close = true;
        before = m;
        if (f == p.fan) break;
        int at = V;
#pragma unroll
        for (int v = V - 1; v >= 0; --v) at = key[v] == m ? v : at;
        const int e = at < V && m != T(kNone) ? sub * E::B + at / E::B * (E::B * L) + at % E::B : 1 << 30;
        const int winner = lanes_min<L>(e);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e == winner && v == at) key[v] = T(kNone);
        const int found = winner < (1 << 30) ? winner : -1;
#pragma unroll
        for (int i = 0; i < kRouteFan / 16; ++i)
            if (i < (p.fan + L - 1) / L && f == i * L + sub) id[i] = found;
    }
    return close;
}

// Renormalised gates: the largest pick (sigmoids: below 0, or 0), the scores' common factor.
template <int L>
__device__ __forceinline__ float largest_pick(const RouteParams &p, const float (&pick)[kRouteFan / 16]) {
    float m = kNone;
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) m = pick[i] > m ? pick[i] : m;
    m = lanes_max<L>(m);
    return p.sigmoid && m > 0.0f ? 0.0f : m;
}

// A pick's score, relative to m where there is one (softmax, and renormalised).
__device__ __forceinline__ float pick_score(const RouteParams &p, float l, float m) {
    return l == kNone       ? 0.0f
           : !p.sigmoid     ? exp_below<float>(l, m)
           : p.renormalize  ? shifted_sigmoid(l, m)
                            : sigmoid_of<float>(l);
}

template <int L, int V>
__global__ __launch_bounds__(kRouteWaves<L> *kWave) void route_kernel(const RouteParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int R = kWave / L;  // tokens of a wave
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, sub = lane % L, row = lane / L;
    const int64_t token = p.first + ((int64_t)blockIdx.x * kRouteWaves<L> + wave) * R + row;
    const bool live = token < p.tokens;
    const int64_t from = live ? token : p.tokens - 1;
    float l[V];
    load_logits<L, V>(p, from, sub, l);
    char *const mine = lds + (int64_t)wave * R * (p.experts + 2 * p.groups) * 8;
    int id[kRouteFan / 16];
    const bool close = pick_experts<float, L, V>(p, l, sub, row, mine, id);
    if (__ballot(close && live)) pick_experts<double, L, V>(p, l, sub, row, mine, id);

    // the scores of the picks, each in its lane
    const int slots = (p.fan + L - 1) / L;
    float s[kRouteFan / 16];
    float m = kNone, sum = 1.0f;  // what the picks' scores are relative to, and divided by
    float pick[kRouteFan / 16];
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) {
        pick[i] = kNone;
        if (i < slots && id[i] >= 0) pick[i] = load_logit(p, from, id[i]);
    }
    if (p.renormalize) {
        m = largest_pick<L>(p, pick);
    } else if (!p.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) m = l[v] > m ? l[v] : m;
        m = lanes_max<L>(m);
        sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += l[v] == kNone ? 0.0f : exp_below<float>(l[v], m);
        sum = lanes_sum<L>(sum);
    }
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) s[i] = pick_score(p, pick[i], m);
    if (p.renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kRouteFan / 16; ++i) sum += s[i];
        sum = lanes_sum<L>(sum);
    }
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) {
        const int f = i * L + sub;
        if (!live || f >= p.fan) continue;
        p.ids[token * p.fan + f] = id[i];
        // (without an expert the sum is 0)
        p.gates[token * p.fan + f] = sum > 0.0f ? p.scale * (s[i] / sum) : 0.0f;
    }
}

// dl of the gates: with the gates' own gradient c_f = scale dgate_f,
//   renormalised:  dl = g_f (c_f - sum_j c_j g_j), g = s / sum of s, times 1 - s for a sigmoid;
//   otherwise:     softmax dl_e = s_e ([e picked] c_e - sum_j c_j s_j), sigmoid dl = c_f s (1 - s).
// Bound by bytes: the logits once, dl once.
template <int L, int V>
__global__ __launch_bounds__(kRouteWaves<L> *kWave) void route_grad_kernel(const RouteParams p) {
    using E = Experts<L, V>;
    constexpr int R = kWave / L;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, sub = lane % L, row = lane / L;
    const int64_t token = p.first + ((int64_t)blockIdx.x * kRouteWaves<L> + wave) * R + row;
    const bool live = token < p.tokens;
    const int64_t from = live ? token : p.tokens - 1;
    const bool dense = !p.sigmoid && !p.renormalize;  // every expert has a gradient
    float l[V];
    float m = kNone, total = 0.0f;
    if (dense) {
        load_logits<L, V>(p, from, sub, l);
#pragma unroll
        for (int v = 0; v < V; ++v) m = l[v] > m ? l[v] : m;
        m = lanes_max<L>(m);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            l[v] = l[v] == kNone ? 0.0f : exp_below<float>(l[v], m);
            total += l[v];
        }
        total = lanes_sum<L>(total);
    }
    const int slots = (p.fan + L - 1) / L;
    int id[kRouteFan / 16];
    float c[kRouteFan / 16], pick[kRouteFan / 16], s[kRouteFan / 16];
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) {
        const int f = i * L + sub;
        id[i] = -1;
        c[i] = 0.0f;
        pick[i] = kNone;
        if (i < slots && f < p.fan) {
            id[i] = p.ids[from * p.fan + f];
            if (id[i] < 0 || id[i] >= p.experts) id[i] = -1;
            if (id[i] >= 0) {
                c[i] = p.scale * p.dgates[from * p.fan + f];
                pick[i] = load_logit(p, from, id[i]);
                if (!(pick[i] > kNone)) id[i] = -1, pick[i] = kNone;  // -inf, NaN
            }
        }
    }
    if (p.renormalize) m = largest_pick<L>(p, pick);
    float weighted = 0.0f, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) {
        s[i] = pick_score(p, pick[i], m);
        sum += s[i];
    }
    if (p.renormalize)
        sum = lanes_sum<L>(sum);
    else
        sum = p.sigmoid ? 1.0f : total;
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) {
        s[i] = sum > 0.0f ? s[i] / sum : 0.0f;  // the gate without its scale
        if (id[i] >= 0) weighted += c[i] * s[i];
    }
    weighted = p.renormalize || !p.sigmoid ? lanes_sum<L>(weighted) : 0.0f;
    float d[kRouteFan / 16];  // dense: c; else dl of the pick
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) {
        const float rest = p.sigmoid && id[i] >= 0 ? sigmoid_of<float>(-pick[i]) : 1.0f;  // 1 - s
        d[i] = id[i] < 0 ? 0.0f : dense ? c[i] : (p.renormalize ? c[i] - weighted : c[i]) * s[i] * rest;
    }
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.0f;
    for (int f = 0; f < p.fan; ++f) {
        int who;
        float value;
        if (L == 16 && f >= 16) {
            who = __shfl(id[1], row * L + f - 16);
            value = __shfl(d[1], row * L + f - 16);
        } else {
            who = __shfl(id[0], row * L + f);
            value = __shfl(d[0], row * L + f);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] += E::at(v, sub) == who ? value : 0.0f;
    }
    if (dense) {
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = l[v] / total * (out[v] - weighted);
        // (a row without an expert: total is 0, and every l)
        if (!(total > 0.0f)) {
#pragma unroll
            for (int v = 0; v < V; ++v) out[v] = 0.0f;
        }
    }
    if (!live) return;
#pragma unroll
    for (int v = 0; v < V; v += E::B) {
        const int e = E::at(v, sub);
        const int64_t at = token * p.experts + e;
        if (E::B == 4 && p.vec) {
            if (e >= p.experts) continue;
            if (p.f32) {
                floatx4 x;
#pragma unroll
                for (int i = 0; i < E::B; ++i) x[i] = out[v + i];
                *reinterpret_cast<floatx4 *>(static_cast<float *>(p.dlogits) + at) = x;
            } else {
                half4 x;
#pragma unroll
                for (int i = 0; i < E::B; ++i) x[i] = (_Float16)out[v + i];
                *reinterpret_cast<half4 *>(static_cast<_Float16 *>(p.dlogits) + at) = x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E::B; ++i) {
                if (e + i >= p.experts) continue;
                if (p.f32)
                    static_cast<float *>(p.dlogits)[at + i] = out[v + i];
                else
                    static_cast<_Float16 *>(p.dlogits)[at + i] = (_Float16)out[v + i];
            }
        }
    }
}

template <int L, int V>
static hipError_t launch(bool grad, const RouteParams &p, hipStream_t s) {
    constexpr int R = kRouteWaves<L> * (kWave / L);  // tokens of a workgroup
    const size_t lds = grad || p.groups == 1 ? 0 : (size_t)R * (p.experts + 2 * p.groups) * 8;
    RouteParams q = p;
    void *args[] = {&q};
    const void *kernel = grad ? reinterpret_cast<const void *>(route_grad_kernel<L, V>)
                              : reinterpret_cast<const void *>(route_kernel<L, V>);
    // a launch holds fewer than 2^32 threads
    constexpr int64_t kMost = ((int64_t(1) << 32) - 1) / (kRouteWaves<L> * kWave);
    for (int64_t at = 0, all = (p.tokens + R - 1) / R; at < all; at += kMost) {
        q.first = at * R;
        const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)std::min(kMost, all - at)), dim3(kRouteWaves<L> * kWave),
                                             args, lds, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

static hipError_t launch_by_experts(bool grad, const RouteParams &p, hipStream_t s) {
    if (p.experts <= 16) return launch<16, 1>(grad, p, s);
    if (p.experts <= 32) return launch<16, 2>(grad, p, s);
    if (p.experts <= 64) return launch<16, 4>(grad, p, s);
    if (p.experts <= 128) return launch<16, 8>(grad, p, s);
    if (p.experts <= 256) return launch<16, 16>(grad, p, s);
    if (p.experts <= 512) return launch<64, 8>(grad, p, s);
    if (p.experts <= 1024) return launch<64, 16>(grad, p, s);
    return launch<64, 32>(grad, p, s);
}

hipError_t launch_route(const RouteParams &p, hipStream_t s) { return launch_by_experts(false, p, s); }
hipError_t launch_route_grad(const RouteParams &p, hipStream_t s) { return launch_by_experts(true, p, s); }

}  // namespace gemm_f16
