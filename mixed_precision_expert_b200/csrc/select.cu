// The choice of experts from router logits (mpe_select_experts) and the
// experts' mean routing scores (mpe_expert_importance).
#include <cfloat>
#include <cstdarg>
#include <cstdio>

#include "internal.h"
#include "opcheck.h"

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

// Lane `lane`'s EPL consecutive values of a row of E (-inf past its end).
// `wide`: the row starts on a 16-byte boundary and E is a multiple of EPL, so
// that a lane's values are one aligned run, all inside or all outside.
template <typename T, int EPL>
__device__ __forceinline__ void load_row(const T* row, int E, bool wide, int lane, float (&x)[EPL]) {
    const int e0 = lane * EPL;
    constexpr int kBytes = EPL * (int)sizeof(T);
    if constexpr (kBytes % 16 == 0) {
        if (wide) {
            if (e0 < E) {
                constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
                    T t[kPer];
                    memcpy(t, &v, 16);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) x[i * kPer + j] = as_float(t[j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) x[i] = -INFINITY;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = e0 + i < E ? as_float(row[e0 + i]) : -INFINITY;
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
    int wide;
};

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

// ---- the choice, one warp a token -----------------------------------------
// Lane l holds the keys of experts l EPL .. l EPL + EPL - 1. The k-th largest of
// the lanes' largest keys is a threshold that at least k keys reach, and few
// others (ten on the average for k = 8 of 256): the keys that reach it are moved
// to one lane each, in the experts' order, and each lane counts the keys ahead of
// its own. That costs a few instructions a key where k searches for a maximum
// cost as many each. Where fewer than 2k lanes hold keys, or more than 32 keys
// reach the threshold, k searches it is.
//
// Error of the float32 keys. Softmax: a term e^-d, d = m - l, carries the
// exponential's 2 ulp (4 units of 2^-24) and the rounding of d (d units). The
// sum of the terms adds EPL - 1 + 5 roundings and the mean of d under the
// scores, which is at most their entropy, ln 1024 < 7; reciprocal and product
// add 2; d s < 1/2 in the numerator. With s <= 1 that is at most EPL + 24 units.
// Sigmoid: the fast exponential is off by 2 + 1.2 |l| ulp, which s (1 - s) <=
// e^-|l| turns into less than 2^-23 of the score; an addition and a reciprocal
// of 1 ulp: below 2^-21. Adding the bias rounds by 2^-24 |key|. Keys (or sums of
// two) further apart than the errors of both are in float64's order; nearer
// ones, of which a sigmoid with a bias has about one row in 1000, take
// select_exact, as do rows with a NaN or an infinity in the way.
constexpr int kSelWarps = 4;

// The two largest values of several, in order.
__device__ __forceinline__ void push2(float& m1, float& m2, float v) {
    m2 = fmaxf(m2, fminf(m1, v));
    m1 = fmaxf(m1, v);
}

template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kSelWarps) k_select(const SelectArgs a) {
    __shared__ float s_key[kSelWarps][32];
    __shared__ int s_id[kSelWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = (gridDim.x * blockDim.x) >> 5;
    const int e0 = lane * EPL;
    const bool limited = a.keep < a.n_groups;
    const bool sums = limited && a.group_score == MPE_GROUP_TOP2;
    const bool softmax = a.score == MPE_SCORE_SOFTMAX;
    const bool whole = softmax && (a.bias || sums || !a.renorm);  // the softmax's own sum is needed
    const int gs = a.E / a.n_groups;
    // groups of a power of two of whole lanes: their scores by exchange
    const int group_lanes = gs / EPL;
    const bool by_lanes = gs % EPL == 0 && (group_lanes & (group_lanes - 1)) == 0;
    const float err = softmax ? (EPL + 24) * 0x1p-24f : 0x1p-21f;
    constexpr bool kHold = EPL <= 8;  // the bias stays in registers
    float held[kHold ? EPL : 1];
    bool nan_bias = false;
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float b = e0 + i < a.E ? __ldg(a.bias + e0 + i) : 0.0f;
            nan_bias |= b != b;
            if (kHold) held[i] = b;
        }
        nan_bias = __any_sync(kFull, nan_bias);
    }
    for (int t = blockIdx.x * kSelWarps + warp; t < a.T; t += warps) {
        const T* row = static_cast<const T*>(a.logits) + (size_t)t * a.ld;
        float x[EPL];
        load_row<T, EPL>(row, a.E, a.wide, lane, x);
        // NaN, and +inf under the softmax, make the whole row's weights NaN
        const float most = softmax ? FLT_MAX : INFINITY;
        bool broken = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) broken |= !(x[i] <= most);
        broken = __any_sync(kFull, broken);
        float m = 0.0f, inv = 0.0f;
        if (whole) {
            m = x[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) m = fmaxf(m, x[i]);
            m = warp_top(m);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) sum += x[i] == -INFINITY ? 0.0f : expf(x[i] - m);
            sum = warp_sum(sum);
            inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
        }
        auto score = [&](float l) {
            if (!softmax) return __fdividef(1.0f, 1.0f + __expf(-l));
            return l == -INFINITY ? 0.0f : expf(l - m) * inv;
        };
        float key[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            key[i] = x[i];
            if (a.bias && e0 + i < a.E) key[i] = score(x[i]) + (kHold ? held[i] : __ldg(a.bias + e0 + i));
        }
        // -inf from here on: not to be chosen, by its key or by its group
        bool exact = broken || nan_bias;
        if (limited) {
            float mine = -INFINITY, big = 0.0f;  // this lane's group's score; the largest |key| + |key| in a sum
            bool in;
            if (by_lanes) {
                float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e0 + i < a.E) push2(m1, m2, sums && !a.bias ? score(x[i]) : key[i]);
                for (int o = 1; o < group_lanes; o *= 2) {
                    const float o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
                    push2(m1, m2, o1);
                    m2 = fmaxf(m2, o2);
                }
                mine = m1;
                if (sums && gs > 1) {
                    mine = m1 + m2;
                    big = isfinite(mine) ? fabsf(m1) + fabsf(m2) : 0.0f;
                }
                const int g = lane / group_lanes;
                int rank = 0;
                for (int h = 0; h < a.n_groups; ++h) {
                    const float o = __shfl_sync(kFull, mine, h * group_lanes);
                    rank += o > mine || (o == mine && h < g);
                }
                exact |= __any_sync(kFull, g < a.n_groups && mine != mine);
                in = g < a.n_groups && rank < a.keep;
                if (sums || a.bias) {
                    // the last group kept against the first one dropped
                    const float lo = -warp_top(in ? -mine : -INFINITY);
                    const float hi = warp_top(in || g >= a.n_groups ? -INFINITY : mine);
                    exact |= lo - hi <= 4.0f * err + 0x1p-22f * fmaxf(warp_top(big), fabsf(hi));
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = in ? key[i] : -INFINITY;
            } else {
                // lane g: group g
                for (int g = 0; g < a.n_groups; ++g) {
                    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < EPL; ++i)
                        if ((unsigned)(e0 + i - g * gs) < (unsigned)gs) push2(m1, m2, sums && !a.bias ? score(x[i]) : key[i]);
                    const float b1 = warp_top(m1);
                    float s = b1;
                    if (sums && gs > 1) {
                        const int owner = __ffs(__ballot_sync(kFull, m1 == b1)) - 1;
                        const float b2 = warp_top(lane == owner ? m2 : m1);
                        s = b1 + b2;
                        if (isfinite(s)) big = fmaxf(big, fabsf(b1) + fabsf(b2));
                    }
                    if (lane == g) mine = s;
                }
                int rank = 0;
                for (int g = 0; g < a.n_groups; ++g) {
                    const float o = __shfl_sync(kFull, mine, g);
                    rank += o > mine || (o == mine && g < lane);
                }
                exact |= __any_sync(kFull, lane < a.n_groups && mine != mine);
                in = lane < a.n_groups && rank < a.keep;
                const uint32_t kept = __ballot_sync(kFull, in);
                if (sums || a.bias) {
                    const float lo = -warp_top(in ? -mine : -INFINITY);
                    const float hi = warp_top(in || lane >= a.n_groups ? -INFINITY : mine);
                    exact |= lo - hi <= 4.0f * err + 0x1p-22f * fmaxf(big, fabsf(hi));
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e0 + i < a.E && !((kept >> ((e0 + i) / gs)) & 1u)) key[i] = -INFINITY;
            }
        }
        // after this, lane c has the expert `id` that is number `rank` in the order (k and more: not chosen)
        int id = 0, rank = lane;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = fmaxf(top, key[i]);
        int found = 0;
        if (!exact && 2 * a.k <= __popc(__ballot_sync(kFull, top != -INFINITY))) {
            float rest = top, best = -INFINITY, edge = -INFINITY;
            for (int j = 0; j < a.k; ++j) {
                edge = warp_top(rest);
                if (j == 0) best = edge;
                if (rest == edge) rest = -INFINITY;
            }
            // -inf: lanes met in equal keys, too few are left
            const float tol = a.bias ? 2.0f * err + 0x1p-22f * fmaxf(fabsf(best), fabsf(edge)) : 0.0f;
            if (edge != -INFINITY) {
                edge -= tol;
                int n = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) n += key[i] >= edge;
                int at = n;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const int y = __shfl_up_sync(kFull, at, o);
                    if (lane >= o) at += y;
                }
                found = __shfl_sync(kFull, at, 31);
                at -= n;
                if (found <= 32) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < EPL; ++i)
                        if (key[i] >= edge) {
                            s_key[warp][at] = key[i];
                            s_id[warp][at++] = e0 + i;
                        }
                    __syncwarp();
                    const float mine = lane < found ? s_key[warp][lane] : -INFINITY;
                    id = lane < found ? s_id[warp][lane] : 0;
                    rank = 0;
                    bool near = false;
                    for (int c = 0; c < found; ++c) {
                        const float o = s_key[warp][c];
                        rank += o > mine || (o == mine && c < lane);
                        near |= fabsf(o - mine) <= tol && c != lane;
                    }
                    if (lane >= found) rank = 32;
                    if (a.bias && __any_sync(kFull, near && lane < found)) {
                        // equal logits with equal biases are equal in float64 too
                        const float l = as_float(row[id]), b = __ldg(a.bias + id);
                        near = false;
                        for (int c = 0; c < found; ++c) {
                            const float o = s_key[warp][c], ol = __shfl_sync(kFull, l, c), ob = __shfl_sync(kFull, b, c);
                            near |= fabsf(o - mine) <= tol && !(l == ol && b == ob);
                        }
                        exact = __any_sync(kFull, near && lane < found);
                    }
                }
            }
        }
        if (!exact && (found == 0 || found > 32)) {
            // k times the largest key, of the lowest lane that has it
            float won = 0.0f;
            rank = lane;
            for (int j = 0; j < a.k && !exact; ++j) {
                const float best = warp_top(top);
                const int src = __ffs(__ballot_sync(kFull, top == best)) - 1;
                exact = best == -INFINITY;
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
                at = __shfl_sync(kFull, at, src & 31);
                if (lane == j) {
                    id = at;
                    won = best;
                }
            }
            if (a.bias && !exact) {
                // neighbours in the order that float32 cannot tell apart
                const float l = lane < a.k ? as_float(row[id]) : 0.0f, b = lane < a.k ? __ldg(a.bias + id) : 0.0f;
                const float pw = __shfl_up_sync(kFull, won, 1), pl = __shfl_up_sync(kFull, l, 1),
                            pb = __shfl_up_sync(kFull, b, 1);
                bool near = false;
                if (lane > 0 && lane < a.k && !(l == pl && b == pb)) near = pw - won <= 2.0f * err + 0x1p-22f * fabsf(pw);
                // and what is left against the last one chosen
                const float lw = __shfl_sync(kFull, won, a.k - 1), ll = __shfl_sync(kFull, l, a.k - 1),
                            lb = __shfl_sync(kFull, b, a.k - 1);
                const float edge = lw - (2.0f * err + 0x1p-22f * fabsf(lw));
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (key[i] >= edge && !(x[i] == ll && __ldg(a.bias + e0 + i) == lb)) near = true;
                exact = __any_sync(kFull, near);
            }
        }
        if (exact) {
            id = select_exact<T>(a, row, lane);
            rank = lane;
        }
        const bool chosen = rank < a.k;
        const float l = chosen ? as_float(row[id]) : -INFINITY;
        // weights: of the chosen logits alone where their sum divides them
        float s = 0.0f;
        if (a.renorm) {
            const float lm = warp_top(l);
            if (chosen && l != -INFINITY) {
                if (softmax) s = expf(l - lm);
                // both factors of e^-lm where the scores may be tiny
                else s = lm < 0.0f ? expf(l - lm) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
            }
            const float sum = warp_sum(s);
            s = sum == 0.0f ? 0.0f : a.scale * (s / sum);
        } else if (chosen) {
            s = a.scale * (softmax ? (l == -INFINITY ? 0.0f : expf(l - m) * inv) : 1.0f / (1.0f + expf(-l)));
        }
        if (chosen) {
            a.ids[(size_t)t * a.k + rank] = id;
            a.w[(size_t)t * a.k + rank] = broken ? NAN : s;
        }
    }
}

template <typename T, int EPL>
cudaError_t launch_select(const SelectArgs& a, int sms, cudaStream_t st) {
    const int64_t want = ((int64_t)a.T + kSelWarps - 1) / kSelWarps, most = (int64_t)sms * 16;
    return launch_pdl(k_select<T, EPL>, dim3((unsigned)(want < most ? want : most)), dim3(32 * kSelWarps), 0, st, a);
}

template <typename T>
cudaError_t launch_select_t(const SelectArgs& a, int sms, cudaStream_t st) {
    if (a.E <= 32) return launch_select<T, 1>(a, sms, st);
    if (a.E <= 64) return launch_select<T, 2>(a, sms, st);
    if (a.E <= 128) return launch_select<T, 4>(a, sms, st);
    if (a.E <= 256) return launch_select<T, 8>(a, sms, st);
    if (a.E <= 512) return launch_select<T, 16>(a, sms, st);
    return launch_select<T, 32>(a, sms, st);
}

// A lane's EPL values are one aligned run of 16-byte pieces inside the row.
bool wide_rows(const void* logits, int32_t type, int64_t ld, int T, int E) {
    int epl = 1;
    while (32 * epl < E) epl *= 2;
    const int sz = type_bytes(type);
    return (epl * sz) % 16 == 0 && E % epl == 0 && aligned(logits, 16) && (T == 1 || (ld * sz) % 16 == 0);
}

// ---- importances ----------------------------------------------------------
struct ImportanceArgs {
    const void* logits;
    int64_t ld;
    float* out;   // [E], or null: this CTA's sums go to part
    float* part;  // [CTAs][E]
    int T, E, score, wide;
};

constexpr int kImpWarps = 16;

// One warp a token, a lane's EPL columns added up in registers over the tokens;
// then over the CTA's warps, and over the CTAs in k_importance_join, always in
// the same order. The fast exponential: 2 + 1.2 d ulp for a score of e^-d.
template <typename T, int EPL>
__global__ void __launch_bounds__(32 * kImpWarps) k_importance(const ImportanceArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ float s_sum[];  // [warps][32 EPL]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.0f;
    for (int t = blockIdx.x * kImpWarps + warp; t < a.T; t += gridDim.x * kImpWarps) {
        float x[EPL];
        load_row<T, EPL>(static_cast<const T*>(a.logits) + (size_t)t * a.ld, a.E, a.wide, lane, x);
        if (a.score == MPE_SCORE_SIGMOID) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) acc[i] += __fdividef(1.0f, 1.0f + __expf(-x[i]));
        } else {
            float m = x[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) m = fmaxf(m, x[i]);
            m = warp_top(m);
            if (m == -INFINITY) m = 0.0f;  // nothing but -inf: scores of 0 (and NaN stays NaN)
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                x[i] = __expf(x[i] - m);
                sum += x[i];
            }
            sum = warp_sum(sum);
            const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
#pragma unroll
            for (int i = 0; i < EPL; ++i) acc[i] = fmaf(x[i], inv, acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) s_sum[(warp * EPL + i) * 32 + lane] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kImpWarps; ++w) s += s_sum[(w * EPL + e % EPL) * 32 + e / EPL];
        if (a.out) a.out[e] = (float)((double)s / a.T);
        else a.part[(size_t)blockIdx.x * a.E + e] = s;
    }
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

// CTAs, each with sums of its own: two to an SM, and more where a warp would
// add up over 256 rows in float32.
int importance_parts(int T) {
    const int most = 296, rows = 256 * kImpWarps;
    const int n = (int)(((int64_t)T + kImpWarps - 1) / kImpWarps);
    const int long_run = (int)(((int64_t)T + rows - 1) / rows);
    return n < most ? n : (long_run > most ? long_run : most);
}

template <typename T, int EPL>
cudaError_t launch_importance(const ImportanceArgs& a, int parts, cudaStream_t st) {
    const size_t smem = (size_t)kImpWarps * 32 * EPL * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(k_importance<T, EPL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_importance<T, EPL>, dim3(parts), dim3(32 * kImpWarps), smem, st, a);
}

template <typename T>
cudaError_t launch_importance_t(const ImportanceArgs& a, int parts, cudaStream_t st) {
    if (a.E <= 32) return launch_importance<T, 1>(a, parts, st);
    if (a.E <= 64) return launch_importance<T, 2>(a, parts, st);
    if (a.E <= 128) return launch_importance<T, 4>(a, parts, st);
    if (a.E <= 256) return launch_importance<T, 8>(a, parts, st);
    if (a.E <= 512) return launch_importance<T, 16>(a, parts, st);
    return launch_importance<T, 32>(a, parts, st);
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
    if (ld < E || ld >= (int64_t)1 << 38)
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

extern "C" int mpe_select_experts(const mpe_select_config* cfg, const void* logits, int32_t type,
                                  int64_t ld, int32_t T, const float* bias, int32_t* ids, float* w,
                                  void* stream) {
    constexpr const char* who = "mpe_select_experts";
    if (!cfg) return report_global_error(MPE_ERR_INVALID, "mpe_select_experts: null config");
    if (T < 0) return report_global_errorf(MPE_ERR_INVALID, "%s: T=%d", who, T);
    const int rc = check_logits(who, logits, type, ld, T, cfg->E, cfg->score);
    if (rc != MPE_OK) return rc;
    if (cfg->n_groups < 1 || cfg->n_groups > MPE_MAX_GROUPS || cfg->E % cfg->n_groups)
        return report_global_errorf(MPE_ERR_INVALID, "%s: n_groups=%d (1 .. %d, a divisor of E=%d)", who,
                                    cfg->n_groups, MPE_MAX_GROUPS, cfg->E);
    if (cfg->keep_groups < 1 || cfg->keep_groups > cfg->n_groups)
        return report_global_errorf(MPE_ERR_INVALID, "%s: keep_groups=%d of %d", who, cfg->keep_groups,
                                    cfg->n_groups);
    if (cfg->group_score != MPE_GROUP_MAX && cfg->group_score != MPE_GROUP_TOP2)
        return report_global_errorf(MPE_ERR_INVALID, "%s: bad group_score %d", who, cfg->group_score);
    if (cfg->k < 1 || cfg->k > MPE_MAX_TOPK || cfg->k > cfg->keep_groups * (cfg->E / cfg->n_groups))
        return report_global_errorf(MPE_ERR_INVALID, "%s: k=%d (1 .. %d, at most the %d experts kept)", who,
                                    cfg->k, MPE_MAX_TOPK, cfg->keep_groups * (cfg->E / cfg->n_groups));
    if ((int64_t)T * cfg->k > MPE_MAX_ASSIGNMENTS)
        return report_global_errorf(MPE_ERR_INVALID, "%s: T*k=%lld above %d", who,
                                    (long long)T * cfg->k, MPE_MAX_ASSIGNMENTS);
    if (T == 0) return MPE_OK;
    if (!ids || !w) return report_global_errorf(MPE_ERR_INVALID, "%s: null output", who);
    if (!aligned(ids, 4) || !aligned(w, 4) || !aligned(bias, 4))
        return report_global_errorf(MPE_ERR_INVALID, "%s: ids, w or bias not aligned to 4 bytes", who);
    SelectArgs a{logits, ld, bias, ids, w, T, cfg->E, cfg->k, cfg->score, cfg->n_groups, cfg->keep_groups,
                 cfg->group_score, cfg->renormalize != 0, cfg->scale, wide_rows(logits, type, ld, T, cfg->E)};
    const int sms = current_sm_count();
    if (sms <= 0) return report_global_errorf(MPE_ERR_CUDA, "%s: no current device", who);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return launched(who, type == MPE_TYPE_F32    ? launch_select_t<float>(a, sms, st)
                         : type == MPE_TYPE_BF16 ? launch_select_t<__nv_bfloat16>(a, sms, st)
                                                 : launch_select_t<__half>(a, sms, st));
}

extern "C" size_t mpe_expert_importance_workspace(int32_t T, int32_t E) {
    if (T < 1 || E < 1 || E > MPE_MAX_EXPERTS) return 0;
    const int parts = importance_parts(T);
    return parts > 1 ? (size_t)parts * E * sizeof(float) : 0;
}

extern "C" int mpe_expert_importance(const void* logits, int32_t type, int64_t ld, int32_t T, int32_t E,
                                     int32_t score, float* p_out, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    constexpr const char* who = "mpe_expert_importance";
    if (T < 1) return report_global_errorf(MPE_ERR_INVALID, "%s: T=%d", who, T);
    const int rc = check_logits(who, logits, type, ld, T, E, score);
    if (rc != MPE_OK) return rc;
    if (!p_out || !aligned(p_out, 4))
        return report_global_errorf(MPE_ERR_INVALID, "%s: p_out null or not aligned to 4 bytes", who);
    const size_t need = mpe_expert_importance_workspace(T, E);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return report_global_errorf(MPE_ERR_INVALID, "%s: the workspace needs %zu bytes, 16-byte aligned", who,
                                    need);
    const int parts = importance_parts(T);
    ImportanceArgs a{logits, ld, parts > 1 ? nullptr : p_out, static_cast<float*>(workspace), T, E, score,
                     wide_rows(logits, type, ld, T, E)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = type == MPE_TYPE_F32    ? launch_importance_t<float>(a, parts, st)
                    : type == MPE_TYPE_BF16 ? launch_importance_t<__nv_bfloat16>(a, parts, st)
                                            : launch_importance_t<__half>(a, parts, st);
    if (e == cudaSuccess && parts > 1)
        e = launch_pdl(k_importance_join, dim3((E + 31) / 32), dim3(1024), 0, st, (const float*)a.part, parts, E,
                       T, p_out);
    return launched(who, e);
}
