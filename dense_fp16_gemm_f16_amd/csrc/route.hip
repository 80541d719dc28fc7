// Routing to experts: the ids and gates of each token's experts from its logits, and the
// gradient of the gates.
//
//   s = softmax(l) or sigmoid(l);  key = s + bias, or l without one
//   expert groups: the top_groups of them with the largest key, or sum of two largest s + bias
//   ids = the fan largest keys in the open groups, in order, ties to the lowest index
//   gates = scale s[ids], or scale s[ids] / sum of s[ids]
//
// A row of 16 lanes takes a token (64 lanes past 256 experts), V logits a lane in registers;
// a reduction over a row is four rotations within it.  Up to 256 experts and 16 picks the candidates
// are sorted at once (sort_candidates); else each pick is one such reduction for the largest key and
// one for its lowest index.
// Bound by the vector unit's issue: 16384 tokens, 8 of 256 experts in 4 of 8 groups, take 15.6 to 17.3 us
// for 17.8 MB; a wave of four tokens issues 1440 vector instructions, which fill 76% of the cycles.
//
// The choice is that of the formula in 64 bits, so which experts a token gets does not hang on
// the order of a sum.  Keys are computed in fp32 and the picks made with them; where keys that
// decide (neighbours in the order, or the last one in and the first one out) are closer than
// their rounding errors, the picks in question get their keys in 64 bits and are put in order.
// Without a bias the order is that of the logits and exact.
#include "route.h"

#include <algorithm>

#include "fused.h"

namespace gemm_f16 {

// Waves of a workgroup: with expert groups a wave keeps its tokens' keys in LDS, 64 KB at most
// for all.
template <int L>
constexpr int kRouteWaves = L == 16 ? 4 : 2;

// A move within rows of 16 lanes.  Every lane of the wave has to take part: what an inactive
// lane holds comes out as 0.
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
// (none of them is a NaN)
__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return __builtin_fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ double smaller(double a, double b) { return a < b ? a : b; }

template <int L, class T>
__device__ __forceinline__ T lanes_max(T x) {
    return lanes_reduce<L>(x, [](T a, T b) { return larger(a, b); });
}

// The largest of a lane's values, as a tree.
template <int V, class T>
__device__ __forceinline__ T largest_of(const T (&x)[V]) {
    T y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = x[v];
#pragma unroll
    for (int d = 1; d < V; d *= 2)
#pragma unroll
        for (int v = 0; v + d < V; v += 2 * d) y[v] = larger(y[v], y[v + d]);
    return y[0];
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
constexpr float kMost = __FLT_MAX__;

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

// exp for keys: in fp32 the hardware's exp2 of a rounded product, relatively off by |x| 2^-24 +
// 2^-23.  A key needs it against 1, where x exp(x) <= 0.37 and x s (1 - s) <= 0.23 make that
// less than 2^-23.
__device__ __forceinline__ float key_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ double key_exp(double x) { return exp(x); }
__device__ __forceinline__ float inverse_of(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double inverse_of(double x) { return 1.0 / x; }

// What a choice goes by, in T: among the experts, or (`sums`) for groups valued by a sum.
template <class T, int L, int V>
struct Keys {
    T key[V];  // -inf: never chosen
    T share;   // softmax: the largest score, 1 / sum of exp(l - m)

    __device__ __forceinline__ void init(const RouteParams &p, const float (&l)[V], int sub, bool sums) {
        using E = Experts<L, V>;
        share = T(1);
        const bool by_score = p.bias != nullptr;
        if (!by_score && !sums) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = T(l[v]);
            return;
        }
        if (p.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = inverse_of(T(1) + key_exp(-T(l[v])));
        } else {
            const float m = lanes_max<L>(largest_of<V>(l));
            T sum = T(0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                key[v] = l[v] == kNone ? T(0) : l[v] == m ? T(1) : key_exp(T(l[v]) - T(m));
                sum += key[v];
            }
            share = inverse_of(lanes_sum<L>(sum));
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] *= share;
        }
#pragma unroll
        for (int v = 0; v < V; v += E::B) {
            float bias[E::B];
            const int e = E::at(v, sub);
#pragma unroll
            for (int i = 0; i < E::B; ++i) bias[i] = 0.0f;
            if (by_score) {
                if (E::B == 4 && p.bias_vec) {
                    const floatx4 x = e < p.experts ? *reinterpret_cast<const floatx4 *>(p.bias + e) : floatx4{};
#pragma unroll
                    for (int i = 0; i < E::B; ++i) bias[i] = x[i];
                } else {
#pragma unroll
                    for (int i = 0; i < E::B; ++i)
                        if (e + i < p.experts) bias[i] = p.bias[e + i];
                }
            }
#pragma unroll
            for (int i = 0; i < E::B; ++i) {
                const T k = key[v + i] + T(bias[i]);
                key[v + i] = l[v + i] == kNone || !(k == k) ? T(kNone) : k;
            }
        }
    }

    // What two fp32 scores can be off by against each other.  A sigmoid: 2^-24.9 by its exp (see
    // key_exp), 2^-24 by its sum and 2^-23 by its reciprocal, less than 2^-22 for each of the
    // two.  A softmax's shares as much relative to the largest, and its sum, which all scores
    // share, is off by less than 2^-18 of itself.  Keys' own roundings come on top (kKeyError).
    __device__ __forceinline__ float error(const RouteParams &p) const { return p.sigmoid ? 0x1p-21f : 0x1p-17f * (float)share; }
};

constexpr float kKeyError = 0x1.1p-23f;  // of a key: both roundings of a comparison, 2^-24 each

// The open groups of the wave's tokens, a bit each, the same in all lanes of a token.  A
// group's value is its largest key, or the sum of its two largest; lane g of a token takes
// group g, from the keys in LDS (a pad per group keeps the lanes on different banks).  close:
// the last group in and some other one are within `error` and their keys' roundings (negative:
// exact).
template <class T, int L, int V>
__device__ __forceinline__ uint64_t open_groups(const RouteParams &p, const Keys<T, L, V> &k, int sub, int row, char *lds, T error,
                                                bool &close) {
    using E = Experts<L, V>;
    const int per = p.experts / p.groups;
    const float inv_per = 1.0f / (float)per;
    T *const keys = reinterpret_cast<T *>(lds) + (int64_t)row * (p.experts + 2 * p.groups);
    T *const value = keys + p.experts + p.groups;
    wave_lds_fence();
    T size = T(1);
    // a group's value from its two largest (one with one expert left counts that one alone)
    auto worth = [&](T first, T second) {
        if (second != T(kNone))
            size = larger(size, larger(larger(first, -first), larger(second, -second)));
        else if (first != T(kNone))
            size = larger(size, larger(first, -first));
        if (p.group_top != 2 || second == T(kNone)) return first;
        const T sum = first + second;
        // Past fp32's range (a bias of its lowest value, say) it stays finite: -inf would be a group
        // of no experts.  Such sums are close to one another and told apart in 64 bits.
        if constexpr (sizeof(T) == 4) return __builtin_amdgcn_fmed3f(sum, -kMost, kMost);
        return sum;
    };
    if (L == 16 && V >= 4 && per >= 4 && per <= 64 && (per & (per - 1)) == 0) {
        // groups of 1, 2, 4, 8 or 16 lanes' neighbours: in registers, each lane of a group
        // meeting the others (256 experts in 8 groups: 2 us less than from LDS)
#pragma unroll
        for (int v = 0; v + 3 < V; v += 4) {
            T first = T(kNone), second = T(kNone);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const T x = k.key[v + i];
                second = larger(second, smaller(first, x));
                first = larger(first, x);
            }
            auto meet = [&](T f, T s) {
                second = larger(smaller(first, f), larger(second, s));
                first = larger(first, f);
            };
            if (per >= 8) meet(rot<0xb1>(first), rot<0xb1>(second));     // the lane next to this one
            if (per >= 16) meet(rot<0x4e>(first), rot<0x4e>(second));    // the other pair of four
            if (per >= 32) meet(rot<0x141>(first), rot<0x141>(second));  // the other four of eight
            if (per >= 64) meet(rot<0x140>(first), rot<0x140>(second));  // the other half of the row
            const int e = E::at(v, sub);
            if (e < p.experts && (e & (per - 1)) == 0) value[group_of(e, inv_per)] = worth(first, second);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = E::at(v, sub);
            if (e < p.experts) keys[e + group_of(e, inv_per)] = k.key[v];
        }
        wave_lds_fence();
        for (int g = sub; g < p.groups; g += L) {
            T first = T(kNone), second = T(kNone);
            const T *q = keys + g * (per + 1);
#pragma unroll 8
            for (int i = 0; i < per; ++i) {
                const T x = q[i];
                second = larger(second, smaller(first, x));
                first = larger(first, x);
            }
            value[g] = worth(first, second);
        }
    }
    wave_lds_fence();
    // (two keys' roundings on each side, and the sums', of up to twice their size)
    if (error >= T(0)) error += T(4) * T(kKeyError) * lanes_max<L>(size);
    uint64_t mine = 0;  // of this lane's groups
    for (int g = sub; g < p.groups; g += L) {
        const T x = value[g];
        int rank = 0;
        bool near = false;
#pragma unroll 8
        for (int o = 0; o < p.groups; ++o) {
            const T y = value[o], d = x > y ? x - y : y - x;
            rank += y > x || (y == x && o < g);
            near = near || (o != g && d <= error);
        }
        const bool open = rank < p.top_groups && x != T(kNone);
        mine |= (uint64_t)open << g;
        close = close || (open && rank == p.top_groups - 1 && near);
    }
    const auto any = [](int a, int b) { return a | b; };
    const uint32_t lo = (uint32_t)lanes_reduce<L>((int)(uint32_t)mine, any);
    const uint32_t hi = p.groups > 32 ? (uint32_t)lanes_reduce<L>((int)(uint32_t)(mine >> 32), any) : 0;
    return (uint64_t)hi << 32 | lo;
}

template <class T, int L, int V>
__device__ __forceinline__ void close_groups(const RouteParams &p, Keys<T, L, V> &k, uint64_t open, int sub) {
    using E = Experts<L, V>;
    const int per = p.experts / p.groups;
    const float inv_per = 1.0f / (float)per;
    auto is_open = [&](int v) { return ((open >> (group_of(E::at(v, sub), inv_per) & 63)) & 1) != 0; };
    if (E::B == 4 && per % 4 == 0) {  // four neighbours are in one group
#pragma unroll
        for (int v = 0; v + 3 < V; v += 4) {
            const bool in = is_open(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) k.key[v + i] = in ? k.key[v + i] : T(kNone);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) k.key[v] = is_open(v) ? k.key[v] : T(kNone);
    }
}

// A bound from below of the fan-th largest key of a token of 16 lanes: the fan-th largest among
// the largest keys of 32 disjoint sets, two of a lane: its even and odd values, or (HALVES) its
// first and second half.
template <bool HALVES, int V>
__device__ __forceinline__ float lower_bound(const float (&key)[V], int fan) {
    float part[2][V / 2];
#pragma unroll
    for (int v = 0; v < V; ++v) part[HALVES ? v / (V / 2) : v % 2][HALVES ? v % (V / 2) : v / 2] = key[v];
    const float x = largest_of<V / 2>(part[0]), y = largest_of<V / 2>(part[1]);
    int over_x = y > x, over_y = x > y;  // sets with a larger one
    static_range<1, 16>([&](auto r_c) {
        const float a = rot<0x120 + decltype(r_c)::value>(x), b = rot<0x120 + decltype(r_c)::value>(y);
        over_x += (a > x) + (b > x);
        over_y += (a > y) + (b > y);
    });
    const float least = smaller(over_x < fan ? x : __builtin_inff(), over_y < fan ? y : __builtin_inff());
    return lanes_reduce<16>(least, [](float a, float b) { return smaller(a, b); });
}

// The candidates of tokens of 16 lanes that want up to 16 experts, in falling order of their
// keys: the f-th in lane f of a token (-1: none left).  Few keys reach lower_bound (less
// `error` and the keys' roundings): of 256 normally distributed ones, for 8 experts, 9, and
// more than 16 for one token in 10^4, in whose wave a second bound is tried.  They go to LDS,
// one to a lane, and each counts those before it.  Unlike picks one after the other this does
// not wait for itself.
// false, and no result: some token has more candidates than lanes.  close: neighbours among a
// token's first fan + 1 are within the error (negative: exact).
template <int V>
__device__ __forceinline__ bool sort_candidates(const RouteParams &p, const Keys<float, 16, V> &k, int sub, int row, bool live,
                                                float error, float2 *slots, bool &close, int &id) {
    using E = Experts<16, V>;
    float key;
    int who;
    if constexpr (V == 1) {
        key = k.key[0];
        who = key > kNone ? sub : (1 << 30) + sub;
    } else {
        int count, all;
        float limit;
        auto within = [&](float bound) {
            limit = error >= 0.0f ? bound - (error + kKeyError * __builtin_fabsf(bound)) : bound;
            count = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) count += k.key[v] > kNone && !(k.key[v] < limit);
            all = lanes_sum<16>(count);
        };
        const float bound = lower_bound<false, V>(k.key, p.fan);
        within(bound);
        if constexpr (V >= 4) {
            if (__ballot(live && all > 16)) within(larger(bound, lower_bound<true, V>(k.key, p.fan)));
        }
        if (__ballot(live && all > 16)) return false;
        // places: the candidates of the lanes before, then this lane's own
        // (shifts right within a row, which bring 0 to its first lanes)
        int at = count;
        at += rot<0x111>(at);
        at += rot<0x112>(at);
        at += rot<0x114>(at);
        at += rot<0x118>(at);
        at -= count;
        float2 *const mine = slots + row * 16;
        wave_lds_fence();
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (k.key[v] > kNone && !(k.key[v] < limit) && at < 16)
                mine[at++] = make_float2(k.key[v], __builtin_bit_cast(float, E::at(v, sub)));
        wave_lds_fence();
        const float2 slot = mine[sub];
        key = sub < all ? slot.x : kNone;
        who = sub < all ? __builtin_bit_cast(int, slot.y) : (1 << 30) + sub;
    }
    int place = 0;
    static_range<1, 16>([&](auto r_c) {
        const float other = rot<0x120 + decltype(r_c)::value>(key);
        const int o = rot<0x120 + decltype(r_c)::value>(who);
        place += other > key || (other == key && o < who);
    });
    const int to = (row * 16 + place) * 4;
    const float sorted = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute(to, __builtin_bit_cast(int, key)));
    const int expert = __builtin_amdgcn_ds_permute(to, who);
    id = expert < p.experts ? expert : -1;
    if (error >= 0.0f) {
        const float next = __shfl(sorted, row * 16 + ((sub + 1) & 15));
        close = sub < p.fan && sub < 15 && next > kNone && sorted - next <= error + kKeyError * __builtin_fabsf(next);
    }
    return true;
}

// Picks in falling order of the keys: the f-th in lane f % L of a token, slot f / L (-1: none
// left), of p.fan of them.  `bounded`: the picks go on while some token's last one in and
// first one out are within `error` and their roundings (L at most), and `close` says that
// neighbours among a token's first p.fan + 1 are.  Returns the picks made.
template <class T, int L, int V>
__device__ __forceinline__ int pick_experts(const RouteParams &p, Keys<T, L, V> &k, int sub, bool live, bool bounded, float error,
                                            bool &close, int (&id)[kRouteFan / 16]) {
    using E = Experts<L, V>;
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) id[i] = -1;
    T before = T(0);
    int f = 0;
    for (;; ++f) {
        if (f >= p.fan && !bounded) break;
        const T m = lanes_max<L>(largest_of<V>(k.key));
        if (bounded) {
            const bool near = f > 0 && m != T(kNone) && before - m <= T(error) + T(kKeyError) * larger(m, -m);
            if (f <= p.fan) close = close || near;
            if (f >= p.fan && (f >= L || !__ballot(live && near))) break;
            before = m;
        }
        int at = V;
#pragma unroll
        for (int v = V - 1; v >= 0; --v) at = k.key[v] == m ? v : at;
        const int e = at < V && m != T(kNone) ? sub * E::B + at / E::B * (E::B * L) + at % E::B : 1 << 30;
        const int winner = lanes_min<L>(e);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e == winner && v == at) k.key[v] = T(kNone);
        const int found = winner < (1 << 30) ? winner : -1;
#pragma unroll
        for (int i = 0; i < kRouteFan / 16; ++i)
            if (f == i * L + sub) id[i] = found;
    }
    return f;
}

// The experts of the wave's tokens, as the formula in 64 bits chooses them.
template <int L, int V>
__device__ __forceinline__ void choose(const RouteParams &p, const float (&l)[V], int sub, int row, bool live, int64_t token, char *lds,
                                       int (&id)[kRouteFan / 16]) {
    // (the rare ways read the logits again: held through the common one they cost registers)
    const bool by_score = p.bias != nullptr, sums = p.groups > 1 && p.group_top == 2;
    Keys<float, L, V> k;
    k.init(p, l, sub, sums);
    const float error = by_score || sums ? k.error(p) : -1.0f;
    uint64_t open = ~uint64_t(0);
    if (p.groups > 1) {
        bool close = false;
        open = open_groups(p, k, sub, row, lds, by_score || sums ? 2.0f * error : -1.0f, close);
        if (__ballot(close && live)) {
            float again[V];
            load_logits<L, V>(p, token, sub, again);
            Keys<double, L, V> exact;
            exact.init(p, again, sub, sums);
            open = open_groups(p, exact, sub, row, lds, -1.0, close);
        }
        if (sums && !by_score) k.init(p, l, sub, false);
        close_groups(p, k, open, sub);
    }
    bool close = false, sorted = false;
    if constexpr (L == 16) {
        __shared__ float2 slots[kRouteWaves<16> * kWave];
        GEMM_POISON_LDS(slots);
        if (p.fan <= 16) {
            sorted = sort_candidates<V>(p, k, sub, row, live, by_score ? error : -1.0f, slots + threadIdx.x / kWave * kWave, close,
                                        id[0]);
            id[1] = -1;
        }
    }
    int made = 16;
    if (!sorted) made = pick_experts(p, k, sub, live, by_score, error, close, id);
    if (!__ballot(close && live)) {
        if (sorted && sub >= p.fan) id[0] = -1;
        return;
    }
    if (sorted || made < L) {
        // The picks made are all that can be in, in an order that may be off: each lane's
        // pick gets its key in 64 bits, and its place among them.
        double m = 0.0, sum = 1.0;
        if (!p.sigmoid) {
            float again[V];
            load_logits<L, V>(p, token, sub, again);
            const float top = lanes_max<L>(largest_of<V>(again));
            sum = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += again[v] == kNone ? 0.0 : exp_below<double>(again[v], top);
            sum = lanes_sum<L>(sum);
            m = top;
        }
        const int mine = sub < made ? id[0] : -1;
        double key = (double)kNone;
        if (mine >= 0) {
            const float x = load_logit(p, token, mine);
            key = (p.sigmoid ? sigmoid_of<double>(x) : exp_below<double>(x, (float)m) / sum) + (double)p.bias[mine];
        }
        int place = 0;
        auto meet = [&](double other, int who) { place += who >= 0 && (other > key || (other == key && who < mine)); };
        if constexpr (L == 16) {
            static_range<1, 16>([&](auto r_c) {
                constexpr int turn = 0x120 + decltype(r_c)::value;
                meet(rot<turn>(key), rot<turn>(mine));
            });
        } else {
            for (int f = 0; f < made; ++f) meet(__shfl(key, row * L + f), __shfl(mine, row * L + f));
        }
        // (lanes without a pick, and picks of none, keep to the end)
        if (mine < 0) place = sub;
        const int moved = __builtin_amdgcn_ds_permute((row * L + place) * 4, mine);
        id[0] = sub < p.fan ? moved : -1;
        return;
    }
    float again[V];
    load_logits<L, V>(p, token, sub, again);
    Keys<double, L, V> exact;
    exact.init(p, again, sub, false);
    if (p.groups > 1) close_groups(p, exact, open, sub);
    pick_experts(p, exact, sub, live, false, 0.0f, close, id);
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
__global__ __launch_bounds__(kRouteWaves<L> *kWave) __attribute__((amdgpu_waves_per_eu(L == 16 || V <= 8 ? 4 : V <= 16 ? 3 : 1))) void route_kernel(const RouteParams p) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int R = kWave / L;  // tokens of a wave
    GEMM_POISON_LDS_BYTES(lds, p.groups > 1 ? kRouteWaves<L> * R * (p.experts + 2 * p.groups) * 8 : 0);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, sub = lane % L, row = lane / L;
    const int64_t token = p.first + ((int64_t)blockIdx.x * kRouteWaves<L> + wave) * R + row;
    const bool live = token < p.tokens;
    const int64_t from = live ? token : p.tokens - 1;
    float l[V];
    load_logits<L, V>(p, from, sub, l);
    char *const mine = lds + (int64_t)wave * R * (p.experts + 2 * p.groups) * 8;
    float m = kNone, sum = 1.0f;  // what the picks' scores are relative to, and divided by
    if (!p.renormalize && !p.sigmoid) {
        m = lanes_max<L>(largest_of<V>(l));
        sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += l[v] == kNone ? 0.0f : exp_below<float>(l[v], m);
        sum = lanes_sum<L>(sum);
    }
    int id[kRouteFan / 16];
    choose<L, V>(p, l, sub, row, live, from, mine, id);

    // the scores of the picks, each in its lane
    const int slots = (p.fan + L - 1) / L;
    float s[kRouteFan / 16], pick[kRouteFan / 16];
#pragma unroll
    for (int i = 0; i < kRouteFan / 16; ++i) {
        pick[i] = kNone;
        if (i < slots && id[i] >= 0) pick[i] = load_logit(p, from, id[i]);
    }
    if (p.renormalize) m = largest_pick<L>(p, pick);
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
        m = lanes_max<L>(largest_of<V>(l));
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
