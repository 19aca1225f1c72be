// The choice of experts from router logits (mpe_select_experts) and the
// experts' mean routing scores (mpe_expert_importance).
#include <cfloat>
#include <cstdarg>
#include <cstdio>

#include "internal.h"
#include "opcheck.h"
#include "tc.cuh"

namespace mpe {

int report_global_errorf(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return report_global_error(code, buf);
}

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }

// A lane's EPL consecutive values from `row` on, the first n of them (-inf after
// those). `wide`: `row` is aligned to the pieces of up to 16 bytes that are loaded.
template <int BYTES>
struct Piece;
template <>
struct Piece<16> { using type = uint4; };
template <>
struct Piece<8> { using type = uint2; };
template <>
struct Piece<4> { using type = uint32_t; };
template <>
struct Piece<2> { using type = uint16_t; };

template <typename T, int EPL>
__host__ __device__ constexpr int piece_bytes() {
    return EPL * (int)sizeof(T) < 16 ? EPL * (int)sizeof(T) : 16;
}

template <typename T, int EPL>
__device__ __forceinline__ void load_row(const T* row, int n, bool wide, float (&x)[EPL]) {
    if (wide) {
        using P = typename Piece<piece_bytes<T, EPL>()>::type;
        constexpr int kPer = (int)(sizeof(P) / sizeof(T));
#pragma unroll
        for (int i = 0; i < EPL; i += kPer) {
            T t[kPer];
            P v;
            const bool all = i + kPer <= n;
            if (all) v = __ldg(reinterpret_cast<const P*>(row + i));
            memcpy(t, &v, sizeof(P));
#pragma unroll
            for (int j = 0; j < kPer; ++j) x[i + j] = all ? as_float(t[j]) : -INFINITY;
            if (!all && i < n) {  // the row's end inside a piece
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (i + j < n) x[i + j] = as_float(row[i + j]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] = i < n ? as_float(row[i]) : -INFINITY;
    }
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <typename V>
__device__ __forceinline__ V warp_max(V v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const V y = __shfl_xor_sync(kFull, v, o);
        v = y > v ? y : v;
    }
    return v;
}

// The largest value over the warp (NaN counts as nothing).
__device__ __forceinline__ float warp_top(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

struct SelectArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    int32_t* ids;
    float* w;
    int T, E, k, score, n_groups, keep, group_score, renorm;
    float scale;
    // lanes: group g (the one group of all experts when every group is kept) has
    // lanes g lanes .. (g + 1) lanes - 1, a power of two, lane i of them its experts
    // i EPL .. i EPL + EPL - 1
    int lanes;
    int wide;  // every lane's run starts where its pieces of up to 16 bytes do
};

__device__ __forceinline__ double score64(double l, double m, double sum, bool softmax) {
    if (!softmax) return 1.0 / (1.0 + exp(-l));
    return l == -INFINITY || sum == 0.0 ? 0.0 : exp(l - m) / sum;
}

// ---- float64 choice -------------------------------------------------------
// The same choice with float64 keys, for the rows whose float32 keys are too
// close together to decide. Returns lane j's expert (j < k).
template <typename V>
__device__ __forceinline__ bool better(V a, int ia, V b, int ib) {
    // NaN ranks lowest, ties go to the lower index
    if (a == a && !(b == b)) return true;
    if (!(a == a) && b == b) return false;
    if (a > b) return true;
    if (a < b) return false;
    return ia < ib;
}

// Best (value, index) over the warp; index -1 stands for nothing.
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const double ov = __shfl_xor_sync(kFull, v, o);
        const int oi = __shfl_xor_sync(kFull, i, o);
        if (oi >= 0 && (i < 0 || better(ov, oi, v, i))) {
            v = ov;
            i = oi;
        }
    }
}

template <typename T>
__device__ __noinline__ int select_exact(const SelectArgs& a, const T* row, int lane) {
    constexpr int kMaxPer = MPE_MAX_EXPERTS / 32;
    const int per = (a.E + 31) / 32;
    double key[kMaxPer];  // expert lane + 32 i
    uint32_t open = 0;    // bit i: may be chosen
    double m = -INFINITY;
    for (int i = 0; i < per; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < a.E ? (double)as_float(row[e]) : -INFINITY;
        if (e < a.E) {
            open |= 1u << i;
            m = key[i] > m ? key[i] : m;
        }
    }
    m = warp_max(m);
    double sum = 0.0;
    for (int i = 0; i < per; ++i) {
        if (!((open >> i) & 1u)) continue;
        if (a.score == MPE_SCORE_SIGMOID) {
            key[i] = 1.0 / (1.0 + exp(-key[i]));
        } else {
            key[i] = key[i] == -INFINITY ? 0.0 : exp(key[i] - m);
            sum += key[i];
        }
    }
    sum = warp_sum(sum);
    for (int i = 0; i < per; ++i) {
        const int e = lane + 32 * i;
        if (!((open >> i) & 1u)) continue;
        if (a.score == MPE_SCORE_SOFTMAX) key[i] = sum == 0.0 ? 0.0 : key[i] / sum;
        if (a.bias) key[i] += (double)a.bias[e];
    }
    // without a bias: scores keep the logits' order, but may meet where logits do not
    auto by_logits = [&] {
        for (int i = 0; i < per; ++i)
            if ((open >> i) & 1u) key[i] = (double)as_float(row[lane + 32 * i]);
    };
    if (!a.bias && a.group_score == MPE_GROUP_MAX) by_logits();
    if (a.keep < a.n_groups) {
        const int gs = a.E / a.n_groups;
        double mine = 0.0;  // lane g: group g's score
        for (int g = 0; g < a.n_groups; ++g) {
            double v = 0.0, s = 0.0;
            int first = -1;
            for (int r = 0; r < (a.group_score == MPE_GROUP_TOP2 && gs > 1 ? 2 : 1); ++r) {
                int b = -1;
                for (int i = 0; i < per; ++i) {
                    const int e = lane + 32 * i;
                    if (e >= a.E || e / gs != g || e == first) continue;
                    if (b < 0 || better(key[i], e, v, b)) {
                        v = key[i];
                        b = e;
                    }
                }
                warp_best(v, b);
                first = b;
                s = r ? s + v : v;
            }
            if (lane == g) mine = s;
        }
        int rank = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const double o = __shfl_sync(kFull, mine, g);
            rank += g != lane && better(o, g, mine, lane);
        }
        const uint32_t kept = __ballot_sync(kFull, lane < a.n_groups && rank < a.keep);
        for (int i = 0; i < per; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((kept >> (e / gs)) & 1u)) open &= ~(1u << i);
        }
    }
    if (!a.bias && a.group_score != MPE_GROUP_MAX) by_logits();
    int id = 0;
    for (int j = 0; j < a.k; ++j) {
        double v = 0.0;
        int b = -1;
        for (int i = 0; i < per; ++i) {
            const int e = lane + 32 * i;
            if (((open >> i) & 1u) && (b < 0 || better(key[i], e, v, b))) {
                v = key[i];
                b = e;
            }
        }
        warp_best(v, b);
        if (lane == (b & 31)) open &= ~(1u << (b >> 5));
        if (lane == j) id = b;
    }
    return id;
}

// Whether this lane's group is kept, by float64 keys: for the rows whose groups'
// float32 scores are too close together to decide. (No NaN in the row.)
template <typename T>
__device__ __noinline__ bool groups_exact(const SelectArgs& a, const T* row, int lane, int group, int e0, int n, double m) {
    const bool softmax = a.score == MPE_SCORE_SOFTMAX;
    const int gs = a.E / a.n_groups;
    double sum = 0.0;
    if (softmax) {
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const double l = (double)as_float(row[e0 + i]);
            sum += l == -INFINITY ? 0.0 : exp(l - m);
        }
        sum = warp_sum(sum);
    }
    double m1 = -INFINITY, m2 = -INFINITY;
    auto push = [&](double v) {
        const double less = m1 < v ? m1 : v;
        m2 = m2 > less ? m2 : less;
        m1 = m1 > v ? m1 : v;
    };
#pragma unroll 4
    for (int i = 0; i < n; ++i)
        push(score64((double)as_float(row[e0 + i]), m, sum, softmax) + (a.bias ? (double)a.bias[e0 + i] : 0.0));
    for (int o = 1; o < a.lanes; o *= 2) {
        const double o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
        push(o1);
        m2 = m2 > o2 ? m2 : o2;
    }
    const double mine = a.group_score == MPE_GROUP_TOP2 && gs > 1 ? m1 + m2 : m1;
    int rank = 0;
    for (int g = 0; g < a.n_groups; ++g) {
        const double o = __shfl_sync(kFull, mine, g * a.lanes);
        rank += o > mine || (o == mine && g < group);
    }
    return group < a.n_groups && rank < a.keep;
}

// This lane's place among the first `found` lanes' experts, by their float64 keys
// (without a bias: by the logits), ties by the index.
template <typename T>
__device__ __noinline__ int rank_exact(const SelectArgs& a, const T* row, int e0, int n, double m, int id, int found) {
    const bool softmax = a.score == MPE_SCORE_SOFTMAX;
    double v = (double)as_float(row[id]);
    if (a.bias) {
        double sum = 0.0;
        if (softmax) {
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const double l = (double)as_float(row[e0 + i]);
                sum += l == -INFINITY ? 0.0 : exp(l - m);
            }
            sum = warp_sum(sum);
        }
        v = score64(v, m, sum, softmax) + (double)__ldg(a.bias + id);
    }
    int rank = 0;
    for (int c = 0; c < found; ++c) {
        const double o = __shfl_sync(kFull, v, c);
        const int oid = __shfl_sync(kFull, id, c);
        rank += o > v || (o == v && oid < id);
    }
    return rank;
}

// ---- the choice, one warp a token -----------------------------------------
// A lane holds EPL experts' keys, in the experts' order over the lanes. The k-th
// largest of the lanes' largest keys is a threshold that at least k keys reach,
// and few others (ten on the average for k = 8 of 256): the keys that reach it
// are moved to one lane each, and each lane counts the keys ahead of its own.
// That costs a few instructions a key where k searches for a maximum cost as many
// each. Where too few lanes hold keys for that, or more than 32 keys reach the
// threshold, k searches it is.
//
// Error of the float32 keys. Softmax: a term e^-d, d = m - l, carries the
// exponential's 2 ulp (4 units of 2^-24) and the rounding of d (d units). The
// sum of the terms adds EPL - 1 + 5 roundings and the mean of d under the
// scores, which is at most their entropy, ln 1024 < 7; reciprocal and product
// add 2; d s < 1/2 in the numerator. With s <= 1 that is at most EPL + 24 units.
// Sigmoid: the fast exponential is off by 2 + 1.2 |l| ulp, which s (1 - s) <=
// e^-|l| turns into less than 2^-23 of the score; an addition and a reciprocal
// of 1 ulp: below 2^-21. Adding the bias rounds by 2^-24 |key|. Keys (or sums of
// two) further apart than the errors of both are in float64's order. Of nearer
// keys, which a sigmoid with a bias has in one row of 1000, the order is found
// again from their float64 values (rank_exact), and which groups stay where those
// are near (groups_exact); rows with a NaN, or with too few keys above -inf, take
// select_exact.
constexpr int kSelWarps = 4;

// The two largest values of several, in order (no NaN).
__device__ __forceinline__ void push2(float& m1, float& m2, float v) {
    m2 = fmaxf(m2, fminf(m1, v));
    m1 = fmaxf(m1, v);
}

__device__ __forceinline__ float fast_rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float one_if_greater(float a, float b) {
    float r;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float fast_exp2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + e^-l)
__device__ __forceinline__ float fast_sigmoid(float l) {
    return fast_rcp(1.0f + fast_exp2(-1.44269504f * l));
}

// The n-th largest of the lanes' values, or less where some are equal (-inf:
// fewer than n are different); `best`: the largest.
__device__ __forceinline__ float nth_top(float v, int n, float& best) {
    best = warp_top(v);
    float r = best;
#pragma unroll 4
    for (int j = 1; j < n; ++j) {
        if (v == r) v = -INFINITY;
        r = warp_top(v);
    }
    return r;
}

// Token t's ids and weights: lane j < k has the expert `id` that is number j, of logit
// l (-inf in the other lanes), so that the sum's order is the experts' rank; lm is the
// largest chosen logit, m and inv the softmax's maximum and 1 / sum where weights are
// not divided by their own.
__device__ __forceinline__ void write_chosen(const SelectArgs& a, int t, int lane, int id, float l, float lm, bool broken,
                                             bool softmax, float m, float inv) {
    const bool chosen = lane < a.k;
    float s = 0.0f;
    if (a.renorm) {  // of the chosen logits alone
        if (chosen && l != -INFINITY) {
            if (softmax) s = expf(l - lm);
            // both factors of e^-lm where the scores may be tiny
            else s = lm < 0.0f ? __fdividef(expf(l - lm), 1.0f + expf(l)) : __fdividef(1.0f, 1.0f + expf(-l));
        }
        const float sum = warp_sum(s);
        s = sum == 0.0f ? 0.0f : a.scale * __fdividef(s, sum);
    } else if (chosen) {
        s = a.scale * (softmax ? (l == -INFINITY ? 0.0f : expf(l - m) * inv) : 1.0f / (1.0f + expf(-l)));
    }
    if (chosen) {
        a.ids[(size_t)t * a.k + lane] = id;
        a.w[(size_t)t * a.k + lane] = broken ? NAN : s;
    }
}

// ---- 16-bit logits, at most 128 experts, no bias, no groups ------------------------------------
// The logit's 19 bits (sign, exponent and 10 bits of bf16 or f16 as a float, in an
// order-preserving form) and the expert's index below them are one integer that no
// other expert has: a lane sorts its own, and the warp's largest is taken k times,
// which settles ties, infinities and NaN on the way. Up to 128 experts (on the device):
// 8192 x 128 bf16 5.2 us, and 8.6 with k_select, whose threshold takes any key; 32768 x
// 128 16.8 and 24.3; but 32768 x 256 31.3 and 25.7, since a lane moves its keys up k times.
constexpr uint32_t kIndexBits = 0x1FFFu;  // above MPE_MAX_EXPERTS

// In 1 comparison for 2 keys, 5 for 4.
template <int EPL>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[EPL]) {
    auto order = [&](int i, int j) {
        const uint32_t hi = max(v[i], v[j]), lo = min(v[i], v[j]);
        v[i] = hi;
        v[j] = lo;
    };
    if constexpr (EPL == 2) order(0, 1);
    if constexpr (EPL == 4) order(0, 1), order(2, 3), order(0, 2), order(1, 3), order(1, 2);
}

template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kSelWarps) k_select16(const SelectArgs a) {
    static_assert(sizeof(T) == 2 && EPL <= 4 && MPE_MAX_EXPERTS <= kIndexBits, "the keys' parts");
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = (gridDim.x * blockDim.x) >> 5;
    const bool softmax = a.score == MPE_SCORE_SOFTMAX;
    const int e0 = lane * EPL, n = max(0, min(EPL, a.E - e0));
    for (int t = blockIdx.x * kSelWarps + warp; t < a.T; t += warps) {
        const T* row = static_cast<const T*>(a.logits) + (size_t)t * a.ld;
        float x[EPL];
        load_row<T, EPL>(row + e0, n, a.wide, x);
        // NaN, and +inf under the softmax, make the row's weights NaN
        const float most = softmax ? FLT_MAX : INFINITY;
        bool broken = false;
        uint32_t v[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            broken |= !(x[i] <= most);
            const uint32_t b = __float_as_uint(x[i] + 0.0f);  // -0 as +0
            const uint32_t up = b ^ (uint32_t)(((int32_t)b >> 31) | (int32_t)0x80000000);
            v[i] = (x[i] == x[i] ? up & ~kIndexBits : 0u) | (kIndexBits - (uint32_t)(e0 + i));
            if (i >= n) v[i] = 0u;
        }
        broken = __any_sync(kFull, broken);
        sort_descending<EPL>(v);
        uint32_t mine = 0u, first = 0u;
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const uint32_t best = __reduce_max_sync(kFull, v[0]);
            if (v[0] == best) {
#pragma unroll
                for (int i = 0; i + 1 < EPL; ++i) v[i] = v[i + 1];
                v[EPL - 1] = 0u;
            }
            if (lane == j) mine = best;
            if (j == 0) first = best;
        }
        auto logit = [](uint32_t u) {
            return __uint_as_float(u & 0x80000000u ? (u ^ 0x80000000u) & ~kIndexBits : ~u & ~kIndexBits);
        };
        const float lm = logit(first);
        float inv = 0.0f;
        if (softmax && !a.renorm) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) sum += x[i] == -INFINITY ? 0.0f : expf(x[i] - lm);
            sum = warp_sum(sum);
            inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
        }
        write_chosen(a, t, lane, (int)(kIndexBits - (mine & kIndexBits)), lane < a.k ? logit(mine) : -INFINITY, lm, broken,
                     softmax, lm, inv);
    }
}

template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kSelWarps, EPL <= 8 ? 8 : EPL == 16 ? 5 : 3) k_select(const SelectArgs a) {
    __shared__ __align__(16) float s_key[kSelWarps][32];
    __shared__ int s_id[kSelWarps][32], s_found[kSelWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = (gridDim.x * blockDim.x) >> 5;
    const bool limited = a.keep < a.n_groups;
    const bool sums = limited && a.group_score == MPE_GROUP_TOP2;
    const bool softmax = a.score == MPE_SCORE_SOFTMAX;
    const bool whole = softmax && (a.bias || sums || !a.renorm);  // the softmax's own sum is needed
    const int gs = limited ? a.E / a.n_groups : a.E;
    const int group = lane / a.lanes;
    const int from = (lane & (a.lanes - 1)) * EPL;  // in the group
    const int e0 = group * gs + from;
    const int n = group * gs < a.E ? max(0, min(EPL, gs - from)) : 0;
    const float err = softmax ? (EPL + 24) * 0x1p-24f : 0x1p-21f;
    // the bias stays in registers, or, where there are too many, in shared memory
    // by lanes (16 a lane from global memory a row: 32768 x 512 in 77 us instead of 45)
    constexpr bool kHold = EPL <= 8;
    float held[kHold ? EPL : 1];
    __shared__ float s_bias[kHold ? 1 : 32 * EPL];
    bool nan_bias = false;
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float b = i < n ? __ldg(a.bias + e0 + i) : -INFINITY;
            nan_bias |= b != b;
            if (kHold) held[i] = b;
            else if (warp == 0) s_bias[i * 32 + lane] = b;
        }
        nan_bias = __any_sync(kFull, nan_bias);
        if (!kHold) __syncthreads();
    }
    for (int t = blockIdx.x * kSelWarps + warp; t < a.T; t += warps) {
        const T* row = static_cast<const T*>(a.logits) + (size_t)t * a.ld;
        float x[EPL];
        load_row<T, EPL>(row + e0, n, a.wide, x);
        // NaN, and +inf under the softmax, make the whole row's weights NaN
        const float most = softmax ? FLT_MAX : INFINITY;
        float total = x[0];  // shows either
#pragma unroll
        for (int i = 1; i < EPL; ++i) total += x[i];
        bool broken = __any_sync(kFull, !(total <= FLT_MAX));
        if (broken) {
            broken = false;
#pragma unroll
            for (int i = 0; i < EPL; ++i) broken |= !(x[i] <= most);
            broken = __any_sync(kFull, broken);
        }
        bool exact = broken || nan_bias;
        // the scores where they are needed, then the keys; -inf: not to be chosen, by its
        // key or by its group
        float key[EPL];
        float m = 0.0f, inv = 0.0f;
        if (whole) {
            m = x[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) m = fmaxf(m, x[i]);
            m = warp_top(m);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                key[i] = x[i] == -INFINITY ? 0.0f : expf(x[i] - m);
                sum += key[i];
            }
            sum = warp_sum(sum);
            inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] *= inv;
        } else if (a.bias || sums) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = fast_sigmoid(x[i]);
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] += kHold ? held[i] : s_bias[i * 32 + lane];
        } else if (!sums) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = x[i];
        }
        if (limited) {
            float m1 = -INFINITY, m2 = -INFINITY;
            if (sums && !a.bias) {
                // by the scores; the choice is by the logits
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    push2(m1, m2, i < n ? key[i] : -INFINITY);
                    key[i] = x[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) push2(m1, m2, key[i]);
            }
            for (int o = 1; o < a.lanes; o *= 2) {
                const float o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
                push2(m1, m2, o1);
                m2 = fmaxf(m2, o2);
            }
            float mine = m1, big = 0.0f;  // the group's score; |key| + |key| of finite keys (infinite: past float32)
            if (sums && gs > 1) {
                mine = m1 + m2;
                big = isfinite(m1) && isfinite(m2) ? fabsf(m1) + fabsf(m2) : 0.0f;
            }
            if (group >= a.n_groups) mine = -INFINITY;
            // every group's score once, in the first of its lanes
            float best, least = nth_top(from == 0 ? mine : -INFINITY, a.keep, best);
            bool in = group < a.n_groups && mine >= least;
            if (__popc(__ballot_sync(kFull, in && from == 0)) != a.keep) {  // equal scores
                int rank = 0;
                for (int g = 0; g < a.n_groups; ++g) {
                    const float o = __shfl_sync(kFull, mine, g * a.lanes);
                    rank += o > mine || (o == mine && g < group);
                }
                in = group < a.n_groups && rank < a.keep;
                least = -warp_top(in ? -mine : -INFINITY);
            }
            exact |= __any_sync(kFull, mine != mine);
            if (sums || a.bias) {
                // The last group kept against the first one dropped. Where no finite keys' sum is past float32,
                // infinite scores are what they seem, and equal ones stay in the groups' order
                const float over = warp_top(in ? -INFINITY : mine);
                big = warp_top(big);
                if (!exact && (big == INFINITY || least - over <= 4.0f * err + 0x1p-22f * fmaxf(big, fabsf(over))))
                    in = groups_exact<T>(a, row, lane, group, e0, n, (double)m);
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = in ? key[i] : -INFINITY;
        }
        // after this, a lane has the expert `id` that is number `rank` in the order (k and more: not chosen)
        int id = 0, rank = lane, found = 0;
        float mine = -INFINITY, l = -INFINITY;  // its key and logit
        bool unclear = false;
        float top = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = fmaxf(top, key[i]);
        if (!exact && 3 * __popc(__ballot_sync(kFull, top != -INFINITY)) >= 4 * a.k) {
            float best, edge = nth_top(top, a.k, best);
            const float tol = a.bias ? 2.0f * err + 0x1p-22f * fmaxf(fabsf(best), fabsf(edge)) : 0.0f;
            edge -= tol;
            // -inf (or NaN) also when the largest key is +inf, or the k-th near the lowest float: padding and
            // dropped groups would reach that
            if (edge > -INFINITY) {
                __syncwarp();  // the last row's are read
                int count = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) count += key[i] >= edge;
                // places in any order: what is equal is ordered by its index below
                if (lane == 0) s_found[warp] = 0;
                s_key[warp][lane] = -INFINITY;
                __syncwarp();
                int at = count ? atomicAdd(&s_found[warp], count) : 0;
                __syncwarp();
                found = s_found[warp];
                if (found <= 32) {
#pragma unroll
                    for (int i = 0; i < EPL; ++i)
                        if (key[i] >= edge) {
                            s_key[warp][at] = key[i];
                            s_id[warp][at++] = e0 + i;
                        }
                    __syncwarp();
                    // keys above this lane's own beyond doubt: one of every two, unless some are equal or near
                    mine = s_key[warp][lane];
                    const float above = mine + tol;
                    id = lane < found ? s_id[warp][lane] : 0;
                    l = a.bias ? as_float(row[id]) : mine;
                    float over = 0.0f;  // counted as floats: a comparison gives 1.0 or 0.0
                    for (int c = 0; c < found; c += 4) {
                        const float4 o = *reinterpret_cast<const float4*>(&s_key[warp][c]);
                        over += one_if_greater(o.x, above) + one_if_greater(o.y, above);
                        over += one_if_greater(o.z, above) + one_if_greater(o.w, above);
                    }
                    rank = (int)over;
                    unclear = __reduce_add_sync(kFull, lane < found ? rank : 0) != found * (found - 1) / 2;
                }
            }
        }
        if (!exact && (found == 0 || found > 32)) {
            // the largest key, of the lowest lane that has it, k times and then while float32 could be wrong about it
            rank = lane;
            found = 0;
            float edge = -INFINITY, tol = 0.0f;
            while (true) {
                const float best = warp_top(top);
                if (found >= a.k && !(best >= edge)) break;
                if (best == -INFINITY || found == 32) {
                    exact = true;
                    break;
                }
                const int src = __ffs(__ballot_sync(kFull, top == best)) - 1;
                int at = 0;
                if (lane == src) {
                    top = -INFINITY;
                    bool taken = false;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        if (!taken && key[i] == best) {
                            taken = true;
                            at = e0 + i;
                            key[i] = -INFINITY;
                        }
                        top = fmaxf(top, key[i]);
                    }
                }
                at = __shfl_sync(kFull, at, src);
                if (lane == found) {
                    id = at;
                    mine = best;
                }
                if (a.bias) tol = fmaxf(tol, 2.0f * err + 0x1p-22f * fabsf(best));
                if (++found == a.k) {
                    if (!a.bias) break;
                    edge = best - tol;
                }
            }
            const float before = __shfl_up_sync(kFull, mine, 1);
            unclear = a.bias && lane > 0 && lane < found && before - mine <= tol;
            l = as_float(row[id]);
        }
        if (!exact && __any_sync(kFull, unclear)) {
            rank = rank_exact<T>(a, row, e0, n, (double)m, id, found);
        }
        if (lane >= found) rank = 32;
        if (exact) {
            id = select_exact<T>(a, row, lane);
            l = as_float(row[id]);
            rank = lane;
        }
        // to the lane of its rank: places among the candidates came in any order
        __syncwarp();
        if (rank < a.k) {
            s_key[warp][rank] = l;
            s_id[warp][rank] = id;
        }
        __syncwarp();
        l = lane < a.k ? s_key[warp][lane] : -INFINITY;
        id = s_id[warp][lane];
        write_chosen(a, t, lane, id, l, warp_top(l), broken, softmax, m, inv);
    }
}

template <typename T, int EPL>
cudaError_t launch_select(const SelectArgs& a, int sms, cudaStream_t st) {
    const int64_t want = ((int64_t)a.T + kSelWarps - 1) / kSelWarps;
    const dim3 grid((unsigned)(want < (int64_t)sms * 8 ? want : (int64_t)sms * 8)), block(32 * kSelWarps);
    if constexpr (sizeof(T) == 2 && EPL <= 4)
        if (!a.bias && a.keep == a.n_groups) return launch_pdl(k_select16<T, EPL>, grid, block, 0, st, a);
    return launch_pdl(k_select<T, EPL>, grid, block, 0, st, a);
}

template <typename T>
cudaError_t launch_select_t(const SelectArgs& a, int epl, int sms, cudaStream_t st) {
    switch (epl) {
        case 1: return launch_select<T, 1>(a, sms, st);
        case 2: return launch_select<T, 2>(a, sms, st);
        case 4: return launch_select<T, 4>(a, sms, st);
        case 8: return launch_select<T, 8>(a, sms, st);
        case 16: return launch_select<T, 16>(a, sms, st);
        case 32: return launch_select<T, 32>(a, sms, st);
        default: return launch_select<T, 64>(a, sms, st);
    }
}

// Experts a lane has when `groups` groups of gs get `lanes` lanes each, a power of
// two: the fewest that fit the warp (at most 64, at E <= 1024: 17 groups of 60 have a
// lane each).
int experts_per_lane(int groups, int gs, int* lanes) {
    for (int epl = 1;; epl *= 2) {
        int n = 1;
        while (n * epl < gs) n *= 2;
        if (n * groups <= 32) {
            *lanes = n;
            return epl;
        }
    }
}

// Whether every lane's run starts at a multiple of its pieces of up to 16 bytes.
bool wide_rows(const void* logits, int32_t type, int64_t ld, int T, int groups, int gs, int epl) {
    const int sz = type_bytes(type), piece = epl * sz < 16 ? epl * sz : 16;
    return aligned(logits, (size_t)piece) && (T == 1 || (ld * sz) % piece == 0) && (groups == 1 || (gs * sz) % piece == 0);
}

// ---- importances ----------------------------------------------------------
struct ImportanceArgs {
    const void* logits;
    int64_t ld;
    float* out;   // [E] (the CTAs are a cluster), or null: this CTA's sums go to part
    float* part;  // [CTAs][E]
    int T, E, score, wide;  // wide: rows are whole, aligned pieces of 16 bytes
};

constexpr int kImpWarps = 16, kImpCluster = 8;

// One warp a token, its columns added up in registers over the tokens; then over
// the CTA's warps, and over the CTAs (in shared memory where they are a cluster,
// else in k_importance_join), always in the same order. Which columns a lane has
// does not matter: pieces of 16 bytes, the warp's next to each other (single values
// where rows are not aligned to that). A lane copies its pieces of the rows to come
// asynchronously into its own part of shared memory, so that enough rows are on
// their way to keep memory busy while a row's maximum and sum go round the warp.
// The fast exponential, off by 2 + 1.2 d ulp for a score of e^-d: what a mean consists
// of are its rows' large scores (65536 x 256: error against float64 2.8e-8, 2.7e-8 with
// float32's own exponential in torch). With expf: 65536 x 256 float32 14.4 -> 17.1 us.
template <typename T, int EPL>
struct ImpRing {
    static constexpr int kRowBytes = 32 * EPL * (int)sizeof(T);
    static constexpr int kDepth = EPL * (int)sizeof(T) >= 16 ? (kRowBytes <= 1024 ? 4 : 2) : 0;  // rows ahead
    static constexpr int kBytes = kImpWarps * (kDepth * kRowBytes > 128 * EPL ? kDepth * kRowBytes : 128 * EPL);
};

// A row's scores added to acc.
template <int EPL>
__device__ __forceinline__ void add_scores(float (&x)[EPL], bool sigmoid, float (&acc)[EPL]) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] += fast_sigmoid(x[i]);
        return;
    }
    float m = x[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, x[i]);
    m = warp_top(m);
    if (m == -INFINITY) m = 0.0f;  // nothing but -inf: scores of 0 (and NaN stays NaN)
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        x[i] = fast_exp2(1.44269504f * (x[i] - m));
        sum += x[i];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : fast_rcp(sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
}

template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kImpWarps) k_importance(const ImportanceArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ __align__(16) uint8_t s_raw[];
    float* s_sum = reinterpret_cast<float*>(s_raw);  // [warps][EPL][32], after the rows
    using R = ImpRing<T, EPL>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int step = (int)gridDim.x * kImpWarps;
    const bool sigmoid = a.score == MPE_SCORE_SIGMOID;
    const T* logits = static_cast<const T*>(a.logits);
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.0f;
    int64_t t = blockIdx.x * kImpWarps + warp;
    constexpr bool kPieced = R::kDepth > 0;
    constexpr int kPer = kPieced ? 16 / (int)sizeof(T) : 1, kPieces = EPL / kPer;
    const bool pieced = kPieced && a.wide;
    if (pieced) {
        constexpr int kDepth = kPieced ? R::kDepth : 1;
        uint8_t* ring = s_raw + (size_t)warp * kDepth * R::kRowBytes;  // [row][piece][lane]
        auto fetch = [&](int64_t row, int slot) {
            if (row < a.T)
#pragma unroll
                for (int p = 0; p < kPieces; ++p)
                    if ((p * 32 + lane) * kPer < a.E)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         smem_u32(ring + slot * R::kRowBytes + (p * 32 + lane) * 16)),
                                     "l"(logits + (size_t)row * a.ld + (p * 32 + lane) * kPer)
                                     : "memory");
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int d = 0; d < kDepth; ++d) fetch(t + (int64_t)d * step, d);
        for (int slot = 0; t < a.T; t += step) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            float x[EPL];
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                T v[kPer];
                const uint4 w = *reinterpret_cast<const uint4*>(ring + slot * R::kRowBytes + (p * 32 + lane) * 16);
                memcpy(v, &w, sizeof(v));
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    x[p * kPer + i] = (p * 32 + lane) * kPer < a.E ? as_float(v[i]) : -INFINITY;
            }
            fetch(t + (int64_t)kDepth * step, slot);  // this lane has read its part of the slot
            add_scores<EPL>(x, sigmoid, acc);
            if (++slot == kDepth) slot = 0;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the sums take the rows' place
    } else {
#pragma unroll 2
        for (; t < a.T; t += step) {
            float x[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                x[i] = i * 32 + lane < a.E ? as_float(logits[(size_t)t * a.ld + i * 32 + lane]) : -INFINITY;
            add_scores<EPL>(x, sigmoid, acc);
        }
    }
    // by column
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        s_sum[warp * 32 * EPL + (pieced ? (i / kPer * 32 + lane) * kPer + i % kPer : i * 32 + lane)] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kImpWarps; ++w) s += s_sum[w * 32 * EPL + e];
        if (!a.out) a.part[(size_t)blockIdx.x * a.E + e] = s;
        else if (gridDim.x == 1) a.out[e] = (float)((double)s / a.T);
        else s_sum[e] = s;  // of column e only this thread reads here
    }
    if (!a.out || gridDim.x == 1) return;
    tc::cluster_sync();
    for (int e = (int)(blockIdx.x * blockDim.x + threadIdx.x); e < a.E; e += (int)(gridDim.x * blockDim.x)) {
        const uint32_t at = smem_u32(&s_sum[e]);
        float s[kImpCluster][1];
#pragma unroll
        for (int r = 0; r < kImpCluster; ++r) tc::peer_load<1>(tc::peer_addr(at, r), s[r]);
        double sum = 0.0;
#pragma unroll
        for (int r = 0; r < kImpCluster; ++r) sum += (double)s[r][0];
        a.out[e] = (float)(sum / a.T);
    }
    tc::cluster_sync();  // no CTA leaves while another reads its sums
}

// out[e] = 1/T sum over the parts: 32 experts a CTA, every 32nd part a warp.
__global__ void __launch_bounds__(1024) k_importance_join(const float* part, int parts, int E, int T, float* out) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ double s_sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    double s = 0.0;
    if (e < E)
#pragma unroll 8
        for (int p = warp; p < parts; p += 32) s += (double)part[(size_t)p * E + e];
    s_sum[warp][lane] = s;
    __syncthreads();
    s = warp_sum(s_sum[lane][warp]);  // of expert `warp`
    if (lane == 0 && blockIdx.x * 32 + warp < E) out[blockIdx.x * 32 + warp] = (float)(s / T);
}

// CTAs, each with sums of its own, and whether they join them in the same launch: one
// for a few tokens; a cluster, whose CTAs read each other's sums, while its four rows
// a warp take no longer than two launches do (device / call back to back, cluster and
// one CTA: 256 x 128 2.9 / 5.2 and 5.4 / 5.5 us, 64 x 256 3.1 / 5.1 and 3.2 / 5.2, 32 x
// 128 2.6 / 5.3 and 1.9 / 5.2; cluster and two launches, with the workspace's
// allocation: 512 x 128 3.3 / 5.2 and 3.3 / 9.6, 512 x 256 bf16 4.2 / 5.2 and 3.9 / 9.6,
// 2048 x 256 7.8 / 8.3 and 4.6 / 9.6); else two to an SM, and more where a warp would
// add up over 256 rows in float32.
struct ImportancePlan {
    int parts;
    bool join;  // in the same launch
};
ImportancePlan importance_plan(int T, int E) {
    const int64_t size = (int64_t)T * E;
    if (T <= 64 && size <= 1 << 14) return {1, true};
    if (T <= 512 && size <= 1 << 18) return {kImpCluster, true};
    const int most = 296, rows = 256 * kImpWarps;
    const int n = (int)(((int64_t)T + kImpWarps - 1) / kImpWarps);
    const int long_run = (int)(((int64_t)T + rows - 1) / rows);
    return {n < most ? n : (long_run > most ? long_run : most), false};
}

template <typename T, int EPL>
cudaError_t launch_importance(const ImportanceArgs& a, int parts, cudaStream_t st) {
    const size_t smem = ImpRing<T, EPL>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(k_importance<T, EPL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts);
    cfg.blockDim = dim3(32 * kImpWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)kImpCluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = a.out && parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_importance<T, EPL>, a);
}

template <typename T>
cudaError_t launch_importance_t(const ImportanceArgs& a, int epl, int parts, cudaStream_t st) {
    switch (epl) {
        case 1: return launch_importance<T, 1>(a, parts, st);
        case 2: return launch_importance<T, 2>(a, parts, st);
        case 4: return launch_importance<T, 4>(a, parts, st);
        case 8: return launch_importance<T, 8>(a, parts, st);
        case 16: return launch_importance<T, 16>(a, parts, st);
        default: return launch_importance<T, 32>(a, parts, st);
    }
}

// Checks that both calls share; 0 or an error code.
int check_logits(const char* who, const void* logits, int32_t type, int64_t ld, int32_t T, int32_t E,
                 int32_t score) {
    if (E < 1 || E > MPE_MAX_EXPERTS)
        return report_global_errorf(MPE_ERR_INVALID, "%s: E=%d not in 1 .. %d", who, E, MPE_MAX_EXPERTS);
    if (score != MPE_SCORE_SOFTMAX && score != MPE_SCORE_SIGMOID)
        return report_global_errorf(MPE_ERR_INVALID, "%s: bad score %d", who, score);
    if (type != MPE_TYPE_F32 && type != MPE_TYPE_BF16 && type != MPE_TYPE_F16)
        return report_global_errorf(MPE_ERR_INVALID, "%s: bad type %d", who, type);
    if (T > 1 && (ld < E || ld >= (int64_t)1 << 38))
        return report_global_errorf(MPE_ERR_INVALID, "%s: ld=%lld for %d experts", who, (long long)ld, E);
    if (T > 0 && !logits) return report_global_errorf(MPE_ERR_INVALID, "%s: null logits", who);
    if (!aligned(logits, (size_t)type_bytes(type)))
        return report_global_errorf(MPE_ERR_INVALID, "%s: logits not aligned to their type", who);
    return MPE_OK;
}

int launched(const char* who, cudaError_t e) {
    if (e == cudaSuccess) return MPE_OK;
    cudaGetLastError();  // reported here, not left for the next call
    return report_global_errorf(MPE_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

}  // namespace
}  // namespace mpe

using namespace mpe;

extern "C" int mpe_select_experts(const mpe_select_args* p, void* stream) {
    constexpr const char* who = "mpe_select_experts";
    if (!p) return report_global_errorf(MPE_ERR_INVALID, "%s: null args", who);
    if (p->T < 0) return report_global_errorf(MPE_ERR_INVALID, "%s: T=%d", who, p->T);
    const int rc = check_logits(who, p->logits, p->type, p->ld, p->T, p->E, p->score);
    if (rc != MPE_OK) return rc;
    if (p->n_groups < 1 || p->n_groups > MPE_MAX_GROUPS || p->E % p->n_groups)
        return report_global_errorf(MPE_ERR_INVALID, "%s: n_groups=%d (1 .. %d, a divisor of E=%d)", who,
                                    p->n_groups, MPE_MAX_GROUPS, p->E);
    if (p->keep_groups < 1 || p->keep_groups > p->n_groups)
        return report_global_errorf(MPE_ERR_INVALID, "%s: keep_groups=%d of %d", who, p->keep_groups, p->n_groups);
    if (p->group_score != MPE_GROUP_MAX && p->group_score != MPE_GROUP_TOP2)
        return report_global_errorf(MPE_ERR_INVALID, "%s: bad group_score %d", who, p->group_score);
    const int open = p->keep_groups * (p->E / p->n_groups);
    if (p->k < 1 || p->k > MPE_MAX_TOPK || p->k > open)
        return report_global_errorf(MPE_ERR_INVALID, "%s: k=%d (1 .. %d, at most the %d experts kept)", who, p->k,
                                    MPE_MAX_TOPK, open);
    if ((int64_t)p->T * p->k > MPE_MAX_ASSIGNMENTS)
        return report_global_errorf(MPE_ERR_INVALID, "%s: T*k=%lld above %d", who, (long long)p->T * p->k,
                                    MPE_MAX_ASSIGNMENTS);
    if (p->T == 0) return MPE_OK;
    if (!p->ids || !p->w) return report_global_errorf(MPE_ERR_INVALID, "%s: null output", who);
    if (!aligned(p->ids, 4) || !aligned(p->w, 4) || !aligned(p->bias, 4))
        return report_global_errorf(MPE_ERR_INVALID, "%s: ids, w or bias not aligned to 4 bytes", who);
    const Block ids(p->ids, 1, (int64_t)p->T * p->k, 0, 4), w(p->w, 1, (int64_t)p->T * p->k, 0, 4);
    const Block logits(p->logits, p->T, p->E, p->ld, type_bytes(p->type));
    auto over_input = [&](const Block& b) {
        return overlap(b, logits) || (p->bias && overlap(b, Block(p->bias, 1, p->E, 0, 4)));
    };
    if (overlap(ids, w) || over_input(ids) || over_input(w))
        return report_global_errorf(MPE_ERR_INVALID, "%s: ids or w overlaps another argument", who);
    const int groups = p->keep_groups < p->n_groups ? p->n_groups : 1, gs = p->E / groups;
    int lanes = 1;
    const int epl = experts_per_lane(groups, gs, &lanes);
    const SelectArgs a{p->logits, p->ld, p->bias, p->ids, p->w, p->T, p->E, p->k, p->score, p->n_groups,
                       p->keep_groups, p->group_score, p->renormalize != 0, p->scale, lanes,
                       wide_rows(p->logits, p->type, p->ld, p->T, groups, gs, epl)};
    const int sms = current_sm_count();
    if (sms <= 0) return report_global_errorf(MPE_ERR_CUDA, "%s: no current device", who);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return launched(who, p->type == MPE_TYPE_F32    ? launch_select_t<float>(a, epl, sms, st)
                         : p->type == MPE_TYPE_BF16 ? launch_select_t<__nv_bfloat16>(a, epl, sms, st)
                                                    : launch_select_t<__half>(a, epl, sms, st));
}

extern "C" size_t mpe_expert_importance_workspace(int32_t T, int32_t E) {
    if (T < 1 || E < 1 || E > MPE_MAX_EXPERTS) return 0;
    const ImportancePlan how = importance_plan(T, E);
    return how.join ? 0 : (size_t)how.parts * E * sizeof(float);
}

extern "C" int mpe_expert_importance(const mpe_importance_args* p, void* stream) {
    constexpr const char* who = "mpe_expert_importance";
    if (!p) return report_global_errorf(MPE_ERR_INVALID, "%s: null args", who);
    if (p->T < 1) return report_global_errorf(MPE_ERR_INVALID, "%s: T=%d", who, p->T);
    const int rc = check_logits(who, p->logits, p->type, p->ld, p->T, p->E, p->score);
    if (rc != MPE_OK) return rc;
    if (!p->p_out || !aligned(p->p_out, 4))
        return report_global_errorf(MPE_ERR_INVALID, "%s: p_out null or not aligned to 4 bytes", who);
    const size_t need = mpe_expert_importance_workspace(p->T, p->E);
    if (need && (!p->workspace || p->workspace_bytes < need || !aligned(p->workspace, 16)))
        return report_global_errorf(MPE_ERR_INVALID, "%s: the workspace needs %zu bytes, 16-byte aligned", who, need);
    const Block out(p->p_out, 1, p->E, 0, 4), logits(p->logits, p->T, p->E, p->ld, type_bytes(p->type));
    const Block ws(p->workspace, 1, (int64_t)need, 0, 1);
    if (overlap(out, logits) || (need && (overlap(ws, logits) || overlap(ws, out))))
        return report_global_errorf(MPE_ERR_INVALID, "%s: p_out or the workspace overlaps another argument", who);
    const ImportancePlan how = importance_plan(p->T, p->E);
    int lanes = 1;
    const int epl = experts_per_lane(1, p->E, &lanes), sz = type_bytes(p->type);
    const bool pieces = aligned(p->logits, 16) && (p->T == 1 || p->ld * sz % 16 == 0) && p->E * sz % 16 == 0;
    const ImportanceArgs a{p->logits, p->ld, how.join ? p->p_out : nullptr, static_cast<float*>(p->workspace), p->T,
                           p->E, p->score, pieces};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = p->type == MPE_TYPE_F32    ? launch_importance_t<float>(a, epl, how.parts, st)
                    : p->type == MPE_TYPE_BF16 ? launch_importance_t<__nv_bfloat16>(a, epl, how.parts, st)
                                               : launch_importance_t<__half>(a, epl, how.parts, st);
    if (e == cudaSuccess && !how.join)
        e = launch_pdl(k_importance_join, dim3((p->E + 31) / 32), dim3(1024), 0, st, (const float*)a.part, how.parts,
                       p->E, p->T, p->p_out);
    return launched(who, e);
}
