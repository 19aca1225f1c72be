// out = act(x w^T + bias) + residual and its gated form (mpe_linear).
#include <cuda.h>

#include <atomic>
#include <cstdio>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "opcheck.h"
#include "tc.cuh"

namespace mpe {
namespace {

// Sticky status of the current device's context-free calls.
__device__ uint32_t g_status;

// Where a result goes and what is done to it on the way.
struct Epilogue {
    const void *bias, *residual;
    void* out;
    int64_t ldr, ldo;
    int M, N;
    int bias_type, out_type, act;
    int vec;  // out and residual rows take runs of 4 values at multiples of 4
};

__device__ __forceinline__ float load_as_float(const void* p, size_t i, int type) {
    if (type == MPE_TYPE_F32) return static_cast<const float*>(p)[i];
    if (type == MPE_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

// 1 / (1 + e^-v). EXACT, for float32 results: expf, and for either sign from e^-|v|. Else
// the fast exponential, which is off by (2 + 1.2 |v|) ulp: 1.2e-5 at most before the
// result underflows, a twentieth of fp16's half step.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float v) {
    if (EXACT) {
        const float e = expf(-fabsf(v));
        return __fdividef(v < 0.0f ? e : 1.0f, 1.0f + e);
    }
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504f * v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// The normal distribution function. EXACT, for float32 results: erfc(-v / sqrt 2) / 2
// (8192 x 2048 x 768 with bias, gelu and residual: 81 us, 61 with the other). Else, for
// x = |v| and t = 1 / (1 + 0.36 x), the tail is t P(t) e^(-x^2 / 2): P is the polynomial
// of degree 6 with the least relative error over x = 0 .. 14, found by reweighted least
// squares (8.8e-7). In float32: 1.2e-6 near 0, and 0.7 x^2 2^-24 from the exponent's
// argument, 8.4e-6 at x = 13. (Abramowitz and Stegun 7.1.26, which has the same form,
// bounds the absolute error alone, which is 26% of the tail at x = 5; the same product
// with a bf16 result: 42.6 us with it, 43.2 with P.)
template <bool EXACT>
__device__ __forceinline__ float normal_cdf(float v) {
    if (EXACT) return 0.5f * erfcf(-0.70710678f * v);
    float t, e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.36f, fabsf(v), 1.0f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-0.72134752f * v * v));
    float p = fmaf(t, 0.0470559f, -0.17976336f);
    p = fmaf(t, p, 0.18095219f);
    p = fmaf(t, p, 0.026550535f);
    p = fmaf(t, p, 0.13971885f);
    p = fmaf(t, p, 0.14177252f);
    p = fmaf(t, p, 0.14371304f);
    const float q = t * p * e;
    return v < 0.0f ? q : 1.0f - q;
}

// The activation of V values: the choice is outside the loop, so that the code of
// each stands here once a call.
template <int V, bool EXACT>
__device__ __forceinline__ void activate(float (&v)[V], int act) {
    if (act == MPE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid<EXACT>(v[i]);
    } else if (act == MPE_ACT_GELU_TANH) {
        // (1 + tanh z) / 2 = 1 / (1 + e^-2z)
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid<EXACT>(1.59576912f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
    } else if (act == MPE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= normal_cdf<EXACT>(v[i]);
    } else if (act == MPE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
    }
}

// Two values of a 16-bit type.
__device__ __forceinline__ float2 unpack2(uint32_t w, int type) {
    if (type == MPE_TYPE_BF16) {
        __nv_bfloat162 v;
        memcpy(&v, &w, 4);
        return __bfloat1622float2(v);
    }
    __half2 v;
    memcpy(&v, &w, 4);
    return __half22float2(v);
}

// Four values of row m from column n on (n a multiple of 4), those below N.
__device__ __forceinline__ void load_run(const Epilogue& e, const void* base, int64_t ld, int m, int n, float (&r)[4]) {
    const size_t at = (size_t)m * ld + n;
    if (e.vec && n + 4 <= e.N) {
        if (e.out_type == MPE_TYPE_F32) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
            r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
            const float2 a = unpack2(v.x, e.out_type), b = unpack2(v.y, e.out_type);
            r[0] = a.x, r[1] = a.y, r[2] = b.x, r[3] = b.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = n + i < e.N ? load_as_float(base, at + i, e.out_type) : 0.0f;
    }
}

// Two values rounded to the output's 16-bit type.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type) {
    uint32_t r;
    if (type == MPE_TYPE_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        memcpy(&r, &v, 4);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        memcpy(&r, &v, 4);
    }
    return r;
}

__device__ __forceinline__ void store_run(const Epilogue& e, int m, int n, const float (&r)[4]) {
    const size_t at = (size_t)m * e.ldo + n;
    if (e.vec && n + 4 <= e.N) {
        if (e.out_type == MPE_TYPE_F32)
            *reinterpret_cast<float4*>(static_cast<float*>(e.out) + at) = make_float4(r[0], r[1], r[2], r[3]);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(e.out) + at) =
                make_uint2(pack2(r[0], r[1], e.out_type), pack2(r[2], r[3], e.out_type));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (n + i >= e.N) break;
            if (e.out_type == MPE_TYPE_F32) static_cast<float*>(e.out)[at + i] = r[i];
            else if (e.out_type == MPE_TYPE_BF16) static_cast<__nv_bfloat16*>(e.out)[at + i] = __float2bfloat16_rn(r[i]);
            else static_cast<__half*>(e.out)[at + i] = __float2half_rn(r[i]);
        }
    }
}

// Outputs n .. n + V - 1 of token m, V = 4 (rows of whole runs) or 1, from the
// product's sums v (and the up projection's, u): what is read for them first, so
// that several outputs' reads are in flight together, then the rest.
template <int V, bool GATED>
struct Output {
    float v[V], u[V], b[V], bu[V], r[V];
    int m, n;

    __device__ __forceinline__ void fetch(const Epilogue& e) {
        if (e.residual && n < e.N) {
            if constexpr (V == 4) load_run(e, e.residual, e.ldr, m, n, r);
            else r[0] = load_as_float(e.residual, (size_t)m * e.ldr + n, e.out_type);
        }
        if (e.bias) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (n + i >= e.N) break;
                b[i] = load_as_float(e.bias, n + i, e.bias_type);
                if (GATED) bu[i] = load_as_float(e.bias, (size_t)e.N + n + i, e.bias_type);
            }
        }
    }
    __device__ __forceinline__ void finish(const Epilogue& e) {
        if (n >= e.N) return;
        if (e.bias) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] += b[i];
                if (GATED) u[i] += bu[i];
            }
        }
        if (e.out_type == MPE_TYPE_F32) activate<V, true>(v, e.act);
        else activate<V, false>(v, e.act);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (GATED) v[i] *= u[i];
            if (e.residual) v[i] += r[i];
        }
        const size_t at = (size_t)m * e.ldo + n;
        if constexpr (V == 4) store_run(e, m, n, v);
        else if (e.out_type == MPE_TYPE_F32) static_cast<float*>(e.out)[at] = v[0];
        else if (e.out_type == MPE_TYPE_BF16) static_cast<__nv_bfloat16*>(e.out)[at] = __float2bfloat16_rn(v[0]);
        else static_cast<__half*>(e.out)[at] = __float2half_rn(v[0]);
    }
};

// ---------------------------------------------------------------------------
// Few tokens: the weights stream once, their rows are the MMA's M
// ---------------------------------------------------------------------------
// One CTA multiplies 128 rows of w (gated: 64 of the gate's and the same outputs'
// 64 of the up projection's) with NT tokens over a share of K; the S CTAs of a
// cluster share K. Each leaves its sums in its own shared memory, and every CTA
// reads those of its part of the tokens from all of them and adds them up in the
// order of the ranks: no workspace, and a result that does not depend on timing
// (sums sent by bulk copies instead: 0.3 to 0.6 us more).
//   warp 0     loads: per step of 64 inputs a box of w (gated: two) and one of x
//   warps 1, 2 MMAs, M = 128, N = NT: one issuing thread each, every second step,
//              an accumulator each (a step takes one thread 0.28 us whatever NT and
//              the number of stages; two overlap: 1 x 128 x 2048 without a split
//              12.5 -> 7.8 us)
//   warps 4-7  tensor memory -> shared memory (all warps, where it is read once)
//   all        sums over the ranks, epilogue
// The tensor cores cut what they add to an accumulator instead of rounding it: the
// error grows by about 10^-9 of the result a value of K, always towards zero
// (measured: 1.6e-5 at K = 14336). So an accumulator starts again every first_chain()
// inputs, and warps 4-7 add the chains up in registers, rounding to nearest.
constexpr int kKStep = 64;
constexpr int kRows = 128;

// Inputs that an accumulator takes: 512 for a float32 result (error 4.8e-7 at K =
// 14336). For a 16-bit one, whose half step is 120 times what 2048 inputs lose, 2048 in
// k_narrow, so that a CTA's share of K is most often one chain, which all warps read at
// its end (512 x 2048 x 7168: 18.2 us, 21.2 with 1024), and in the first chain of
// k_wide, beside which the epilogue of the tile before runs (4096 x 4096 x 4096 with
// bias, silu and residual: 116 us with 1024 inputs, 110 with 2048, 106 with one chain);
// 1024 in k_wide's next ones.
__host__ __device__ constexpr int first_chain(int out_bytes) { return out_bytes == 4 ? 512 : 2048; }
__host__ __device__ constexpr int next_chain(int out_bytes) { return out_bytes == 4 ? 512 : 1024; }

template <int NT>
struct Narrow {
    static constexpr int kThreads = 256;
    static constexpr int kStageBytes = (kRows + NT) * 128;
    static constexpr int kStages = NT == 128 ? 6 : 4;
    // An issuer takes every second step, and so every second stage: with an odd
    // number it would come back to a stage that the other one had in between, and
    // a barrier's parity cannot tell it a phase from the phase before the last.
    static_assert(kStages % 2 == 0, "stages of an issuer");
    static constexpr int kRing = kStages * kStageBytes;
    // the sums take the ring's place after the last step: [token][row]
    static_assert(NT * kRows * 4 <= kRing, "the sums");
    static constexpr int kSmem = 1024 + kRing + 256;
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
    static constexpr int kCols = 2 * NT;  // two accumulators
};

template <int NT, int S, bool GATED>
__global__ void __launch_bounds__(Narrow<NT>::kThreads)
k_narrow(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Epilogue e,
         const int nk, const int chain, const uint32_t idesc) {
    using C = Narrow<NT>;
    static_assert(NT % S == 0, "tokens of a rank");
    constexpr int kOut = GATED ? kRows / 2 : kRows;  // outputs of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    float* part = reinterpret_cast<float*>(ring);
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + C::kRing);
    uint64_t* empty = full + C::kStages;
    uint64_t* acc_full = empty + C::kStages;  // [2]: the accumulator's chain is complete
    uint64_t* acc_empty = acc_full + 2;       // [2]: read by warps 4-7
    uint64_t* have_tmem = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(have_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)tc::cluster_rank() : 0;
    const int n0 = (int)(blockIdx.x / S) * kOut;
    const int m0 = (int)blockIdx.y * NT;
    const int k_first = (int)((int64_t)nk * rank / S), k_last = (int)((int64_t)nk * (rank + 1) / S);
    // token t of the tile's mt is finished by rank t / per
    const int mt = min(NT, e.M - m0);
    const int per = (mt + S - 1) / S;
    const int mine = max(0, min(per, mt - rank * per));

    if (threadIdx.x == 0) {
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(have_tmem, 1);
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0;
            for (int k = k_first; k < k_last; ++k) {
                if (k - k_first >= C::kStages && !mbar_wait_bounded(&empty[s], phase ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = smem_u32(ring + s * C::kStageBytes);
                mbar_arrive_expect_tx(&full[s], (uint32_t)C::kStageBytes);
                tc::load_box(dst, &map_w, kKStep * k, n0, &full[s]);
                if (GATED) tc::load_box(dst + kRows / 2 * 128, &map_w, kKStep * k, e.N + n0, &full[s]);
                tc::load_box(dst + kRows * 128, &map_x, kKStep * k, m0, &full[s]);
                if (++s == C::kStages) s = 0, phase ^= 1u;
            }
            // on a failed wait, time for copies in flight to land
            if (!ok)
                for (const uint64_t t0 = global_ns(); global_ns() - t0 < 1000000ull;) {
                }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        const int x = warp - 1;  // this issuer's accumulator, and which of every two steps it takes
        if (x == 0) {
            // tensor memory is taken after the wait for earlier kernels, and the next
            // kernel may start only when this one has it: neither can block the other
            tc::tmem_alloc(tmem_slot, C::kCols);
            __syncwarp();
            if (lane == 0) {
                griddep_launch_dependents();
                mbar_arrive(have_tmem);
            }
        }
        if (lane == 0) {
            ok = mbar_wait_bounded(have_tmem, 0);
            const uint32_t d = *tmem_slot + (uint32_t)(x * NT);
            const uint64_t desc = tc::smem_desc(smem_u32(ring));
            int s = x, left = chain;  // left: steps of this chain
            uint32_t phase = 0, acc_phase = 1;
            for (int k = k_first + x; k < k_last && ok; k += 2) {
                if (left == 0) {
                    left = chain;
                    acc_phase ^= 1u;
                    if (!mbar_wait_bounded(&acc_empty[x], acc_phase)) {
                        ok = false;
                        break;
                    }
                }
                if (!mbar_wait_spin(&full[s], phase)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint64_t da = desc + (uint64_t)(s * (C::kStageBytes >> 4)), db = da + (kRows * 128 >> 4);
#pragma unroll
                for (int i = 0; i < kKStep / 16; ++i) tc::mma(d, da + 2 * i, db + 2 * i, idesc, left < chain || i > 0);
                tc::commit(&empty[s]);
                s += 2;
                if (s >= C::kStages) s -= C::kStages, phase ^= 1u;
                if (--left == 0 || k + 2 >= k_last) tc::commit(&acc_full[x]);
            }
        }
        __syncwarp();
    }
    // the sums of this share of K: lanes 32 (w % 4) .. of tensor memory, a row a thread
    const int steps = k_last - k_first, n = ((steps + 1) / 2 + chain - 1) / chain;  // chains of accumulator 0
    if (n == 1) {
        // one chain: all warps at its end, w and w + 4 every second 16 tokens
        ok &= mbar_wait_bounded(&acc_full[0], 0);
        if (steps > 1) ok &= mbar_wait_bounded(&acc_full[1], 0);
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after();
        const uint32_t acc = *tmem_slot + ((uint32_t)((warp & 3) * 32) << 16);
        float* to = part + (warp & 3) * 32 + lane;
#pragma unroll 1
        for (int c = (warp >> 2) * 16; c < mt && ok; c += 32) {
            uint32_t v[2][16];
            tc::tmem_load16(acc + (uint32_t)c, v[0]);
            if (steps > 1) tc::tmem_load16(acc + (uint32_t)(NT + c), v[1]);
            tc::tmem_wait();
            tc::tmem_ready(v[0]);
            tc::tmem_ready(v[1]);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float s = __uint_as_float(v[0][i]);
                to[(c + i) * kRows] = steps > 1 ? s + __uint_as_float(v[1][i]) : s;
            }
        }
    } else if (warp >= 4) {
        float sum[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) sum[i] = 0.0f;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
#pragma unroll 1
        for (int c = 0; c < 2 * n && ok; ++c) {
            const int x = c & 1;
            if (x == 1 && (c >> 1) * chain >= steps / 2) break;  // accumulator 1 may have one fewer
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_full[x], (uint32_t)(c >> 1) & 1u));
            if (!ok) break;
            tc::fence_after();
            const uint32_t acc = *tmem_slot + lanes + (uint32_t)(x * NT);
            // at most 64 values on their way at a time
#pragma unroll
            for (int g = 0; g < NT; g += 64) {
                if (g >= mt) break;
                uint32_t v[NT < 64 ? NT / 16 : 4][16];
#pragma unroll
                for (int h = 0; h < 4 && 16 * h < NT; ++h) tc::tmem_load16(acc + (uint32_t)(g + 16 * h), v[h]);
                tc::tmem_wait();
#pragma unroll
                for (int h = 0; h < 4 && 16 * h < NT; ++h) {
                    tc::tmem_ready(v[h]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[g + 16 * h + i] += __uint_as_float(v[h][i]);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[x]);
        }
        // every MMA is done: the ring's place is free
        float* to = part + (warp & 3) * 32 + lane;
#pragma unroll
        for (int i = 0; i < NT; ++i)
            if (i < mt) to[i * kRows] = sum[i];
    }
    ok = __syncthreads_and(ok);
    const uint32_t tbase = *tmem_slot;
    tc::fence_before();
    if (S > 1) {
        tc::cluster_sync();  // every rank's sums are there
    } else {
        __syncthreads();
    }
    if (!ok && lane == 0) set_status(&g_status, MPE_STATUS_WAIT_TIMEOUT);
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_free(tbase, C::kCols);
    }
    // this rank's tokens, four neighbouring outputs of one a thread; one where rows do
    // not start at runs of four, so that a warp's are next to each other
    const float* own = part + rank * per * kRows;
    auto each = [&](auto v_, auto batch_) {
        constexpr int V = decltype(v_)::value, kBatch = decltype(batch_)::value, kRuns = kOut / V;
#pragma unroll 1
        for (int it = threadIdx.x; it < mine * kRuns; it += kBatch * C::kThreads) {
            Output<V, GATED> o[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = it + j * C::kThreads, t = i / kRuns, r = i % kRuns * V;
                o[j].m = m0 + rank * per + t;
                o[j].n = i < mine * kRuns ? n0 + r : e.N;
                if (i < mine * kRuns) o[j].fetch(e);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = min(it + j * C::kThreads, mine * kRuns - 1), t = i / kRuns, r = i % kRuns * V;
                float v[S][V], u[S][V];
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const uint32_t here = smem_u32(own + t * kRows + r), at = S > 1 ? tc::peer_addr(here, (uint32_t)s) : here;
                    tc::peer_load<V>(at, v[s]);
                    if (GATED) tc::peer_load<V>(at + kOut * 4, u[s]);
                }
#pragma unroll
                for (int i2 = 0; i2 < V; ++i2) {
                    o[j].v[i2] = v[0][i2];
                    if (GATED) o[j].u[i2] = u[0][i2];
#pragma unroll
                    for (int s = 1; s < S; ++s) {
                        o[j].v[i2] += v[s][i2];
                        if (GATED) o[j].u[i2] += u[s][i2];
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) o[j].finish(e);
        }
    };
    // NT 16 has one run a thread
    if (e.vec) each(std::integral_constant<int, 4>(), std::integral_constant<int, NT <= 16 ? 1 : 2>());
    else each(std::integral_constant<int, 1>(), std::integral_constant<int, NT <= 16 ? 2 : 4>());
    if (S > 1) tc::cluster_sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Many tokens: tiles of 256 tokens by BN rows of w, a pair of CTAs each
// ---------------------------------------------------------------------------
// The tokens are the MMA's M (128 in each CTA), BN rows of w its N: each CTA
// loads its tokens and half of the rows of w (gated: rank 0 the gate's, rank 1
// the up projection's rows of the same BN / 2 outputs, so that a thread finds
// both in its own accumulator), and rank 0 issues the MMAs for both. A pair
// takes tiles in turn; two accumulators let the MMAs of a tile run while the
// one before is finished.
//   warp 0     loads into a ring of K-steps of 64
//   warps 1, 2 MMAs (rank 0): with BN 256 an issuing thread's MMAs take as long as
//              issuing them, so two take the chains in turn, and what one does
//              between two chains passes while the other's run; with BN 128 two
//              share every chain, every second step and an accumulator each, as in
//              k_narrow
//   warps 4-11 epilogue, 32 tokens and half of the outputs each: a thread has a
//              token's outputs, which go through 2 KB of shared memory a warp, so
//              that global memory is read and written in runs of 64 bytes of a row
// CHAINED (K beyond one chain of first_chain() inputs an accumulator): the epilogue warps
// add every chain to sums in registers, 128 a thread with BN 256: warps 0-3 leave
// theirs to warps 4-11 (setmaxnreg). The accumulator is free again before the
// epilogue begins. Against one chain that costs 2.5 us where a last round of tiles
// leaves the epilogue uncovered (1024 x 4096 x 4096 with bias, silu and residual: 29.8
// -> 32.5 us, 2048 x 2048 x 7168 with bias and gelu: 45.2 -> 47.7), 2 to 4% of many
// rounds (4096 x 4096 x 4096: 96 -> 100, 8192 x 4096 x 14336: 642 -> 656); chains of 2048
// inputs throughout would cost 0.7% less.
template <int BN, bool CHAINED>
struct Wide {
    static constexpr int kStageBytes = 128 * 128 + BN / 2 * 128;
    static constexpr int kStages = BN == 256 ? 6 : 8;
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int kStaging = 8 * 2048;
    static constexpr int kSmem = 1024 + kRing + kStaging + 4 * BN * 4 + 256;
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
    static constexpr int kIssuers = BN == 256 ? 1 : 2;
    static_assert(kStages % kIssuers == 0, "stages of an issuer");
    static constexpr int kCols = 2 * kIssuers * BN;
    static_assert(kCols <= 512, "tensor memory");
    // registers a thread: at the launch, then of warps 0-3 and of warps 4-11
    static constexpr int kRegs = 168, kFewRegs = BN == 256 ? 40 : 72, kManyRegs = BN == 256 ? 232 : 216;
    static_assert(kFewRegs + 2 * kManyRegs <= 3 * kRegs, "a split of what the block has");
};
constexpr int kWideThreads = 384;
constexpr int kTileM = 256;

struct Tiles {
    int m, n;  // tiles of tokens, of outputs
};

// Tile t of the walk: bands of 8 token tiles, in a band one column of tiles after
// the other, so that the tiles in flight share rows of x and of w in L2.
__device__ __forceinline__ void tile_at(const Tiles& g, int64_t t, int& m, int& n) {
    const int64_t band = t / ((int64_t)8 * g.n);
    const int64_t in = t - band * 8 * g.n;
    const int first = (int)band * 8, rows = min(8, g.m - first);
    n = (int)(in / rows);
    m = first + (int)(in - (int64_t)n * rows);
}

// A warp's 32 rows of 64 bytes: 16-byte piece j of row r lies at j ^ (r / 2 % 4), so
// that neither rows nor columns of pieces meet in a bank.
__device__ __forceinline__ uint8_t* staged(uint8_t* base, int r, int j) {
    return base + r * 64 + ((j ^ ((r >> 1) & 3)) << 4);
}

// Single values between the staging rows and global rows m .. m + 31, columns
// n .. (64 bytes' worth), 16 rows at a time, so that loads are in flight together.
template <typename V, bool STORE>
__device__ __forceinline__ void move_values(uint8_t* stage, void* base, int64_t ld, int m, int n, int M, int N, int lane) {
    constexpr int kPer = 16 / (int)sizeof(V), kCols = 64 / (int)sizeof(V);
    constexpr int kRowsAt = 32 / kCols;  // rows in one pass of the warp: 1 or 2
    constexpr int kBatch = 16;
    V* g = static_cast<V*>(base);
    const int c = lane % kCols;
#pragma unroll 1
    for (int r0 = lane / kCols; r0 < 32; r0 += kBatch * kRowsAt) {
        V v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kRowsAt;
            if (STORE) v[i] = reinterpret_cast<const V*>(staged(stage, r, c / kPer))[c % kPer];
            else if (m + r < M && n + c < N) v[i] = g[(size_t)(m + r) * ld + n + c];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kRowsAt;
            if (!STORE) reinterpret_cast<V*>(staged(stage, r, c / kPer))[c % kPer] = v[i];
            else if (m + r < M && n + c < N) g[(size_t)(m + r) * ld + n + c] = v[i];
        }
    }
}

template <int BN, bool GATED, int SZ, bool CHAINED>
__global__ void __launch_bounds__(kWideThreads, 1)
k_wide(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, const Epilogue e,
       const Tiles grid, const int nk, const uint32_t idesc) {  // nk: steps, a multiple of kIssuers
    using C = Wide<BN, CHAINED>;
    constexpr int kOut = GATED ? BN / 2 : BN;  // outputs of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* staging = ring + C::kRing;
    float* s_bias = reinterpret_cast<float*>(staging + C::kStaging);  // [epilogue warps][BN / 2]
    uint64_t* full = reinterpret_cast<uint64_t*>(s_bias + 4 * BN);    // rank 0: both CTAs' boxes of a stage
    uint64_t* empty = full + C::kStages;                              // each CTA: its stage was multiplied
    uint64_t* acc_full = empty + C::kStages;                          // each CTA: [2] accumulator complete
    uint64_t* acc_empty = acc_full + 2;                               // rank 0: [2] read by both CTAs' epilogue warps
    const int chain = CHAINED ? C::kIssuers * next_chain(SZ) / kKStep : nk;  // steps of all issuers
    const int chain0 = CHAINED ? C::kIssuers * first_chain(SZ) / kKStep : nk;
    uint64_t* turn = acc_empty + 2;                                   // rank 0: [2] an issuer's chain is next
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(turn + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank();
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int64_t tiles = (int64_t)grid.m * grid.n;

    if (threadIdx.x == 0) {
        tc::prefetch_map(&map_x);
        tc::prefetch_map(&map_w);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], C::kIssuers);
            mbar_init(&acc_empty[i], 16);
            mbar_init(&turn[i], 1);
        }
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    if (warp == 1) tc::tmem_alloc_pair(tmem_slot, C::kCols);  // after the wait, as in k_narrow
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const uint32_t tbase = *tmem_slot;
    bool ok = true;
    if constexpr (CHAINED) {
        if (warp < 4) tc::fewer_registers<C::kFewRegs>();
        else tc::more_registers<C::kManyRegs>();
    }

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0;
            bool again = false;  // the ring has been filled once
            for (int64_t t = pair; t < tiles && ok; t += pairs) {
                int m, n;
                tile_at(grid, t, m, n);
                const int x_row = m * kTileM + rank * 128;
                const int w_row = GATED ? n * kOut + (rank ? e.N : 0) : n * kOut + rank * (BN / 2);
                for (int k = 0; k < nk; ++k) {
                    if (again && !mbar_wait_bounded(&empty[s], phase ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(ring + s * C::kStageBytes);
                    const uint32_t bar = tc::peer_addr(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * C::kStageBytes);
                    tc::load_box_pair(dst, &map_x, kKStep * k, x_row, bar);
                    tc::load_box_pair(dst + 128 * 128, &map_w, kKStep * k, w_row, bar);
                    if (++s == C::kStages) s = 0, phase ^= 1u, again = true;
                }
            }
            // every stage that was filled has been multiplied: nothing arrives here any more
            for (int i = 0; i < C::kStages && ok; ++i) {
                if (!again && i >= s) break;
                const bool earlier = i >= s;  // filled in the round before this one
                ok = mbar_wait_bounded(&empty[i], earlier ? phase ^ 1u : phase);
            }
            if (!ok)
                for (const uint64_t t0 = global_ns(); global_ns() - t0 < 1000000ull;) {
                }
        }
        __syncwarp();
    } else if (warp <= 2) {
        if (rank == 0 && lane == 0) {
            const int x = warp - 1;
            const uint64_t desc = tc::smem_desc(smem_u32(ring));
            int s = C::kIssuers == 2 ? x : 0, j = 0;  // j: of the chain
            uint32_t phase = 0, acc_phase = 0, turn_phase = 0;
            for (int64_t t = pair; t < tiles && ok; t += pairs) {
                for (int k0 = 0, k1; k0 < nk && ok; k0 = k1, ++j) {
                    const int b = j & 1;
                    k1 = min(nk, k0 + (k0 == 0 ? chain0 : chain));
                    if (C::kIssuers == 1 && b != x) {
                        const int to = s + k1 - k0, round = to / C::kStages;
                        s = to - round * C::kStages, phase ^= (uint32_t)round & 1u;
                        continue;
                    }
                    if (j >= 2) {
                        ok = mbar_wait_spin(&acc_empty[b], acc_phase);
                        if (C::kIssuers == 1 || b == 1) acc_phase ^= 1u;
                    }
                    // the other issuer has seen every stage before this chain's, so that none is a phase behind
                    if (C::kIssuers == 1 && j > 0) {
                        ok = ok && mbar_wait_spin(&turn[x], turn_phase);
                        turn_phase ^= 1u;
                    }
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t d = tbase + (uint32_t)((C::kIssuers == 1 ? x : 2 * b + x) * BN);
                    int k = k0 + (C::kIssuers == 2 ? x : 0);
                    auto multiply = [&] {
                        tc::fence_after();
                        const uint64_t da = desc + (uint64_t)(s * (C::kStageBytes >> 4)), db = da + (128 * 128 >> 4);
#pragma unroll
                        for (int i = 0; i < kKStep / 16; ++i)
                            tc::mma_pair(d, da + 2 * i, db + 2 * i, idesc, k >= k0 + C::kIssuers || i > 0);
                        tc::commit_pair(&empty[s]);
                        s += C::kIssuers;
                        if (s >= C::kStages) s -= C::kStages, phase ^= 1u;
                    };
                    for (; k < (C::kIssuers == 1 ? k1 - 1 : k1); k += C::kIssuers) {
                        if (!mbar_wait_spin(&full[s], phase)) {
                            ok = false;
                            break;
                        }
                        multiply();
                    }
                    if (C::kIssuers == 1) {  // the last step: the other issuer may go on
                        ok = ok && mbar_wait_spin(&full[s], phase);
                        mbar_arrive(&turn[x ^ 1]);
                        if (!ok) break;
                        multiply();
                    }
                    tc::commit_pair(&acc_full[b]);
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        using V = typename std::conditional<SZ == 4, uint32_t, uint16_t>::type;
        constexpr int kChunk = 64 / SZ;  // outputs in a staging row
        constexpr int kHalf = kOut / 2;  // outputs of this warp
        const int q = warp & 3, half = (warp - 4) >> 2;  // lanes 32 q .. of tensor memory
        uint8_t* stage = staging + (warp - 4) * 2048;
        float* bias = s_bias + (warp - 4) * (BN / 2);  // [0, kHalf): of the outputs (the gate's); then the up projection's
        const int row = lane >> 2, piece = lane & 3;   // of the 16-byte moves: rows row + 8 i
        int b = 0;
        uint32_t phase = 0;
        for (int64_t t = pair; t < tiles && ok; t += pairs) {
            int mt, nt;
            tile_at(grid, t, mt, nt);
            const int m = mt * kTileM + rank * 128 + q * 32, n0 = nt * kOut + half * kHalf;
            if (e.bias) {
                for (int i = lane; i < BN / 2; i += 32) {
                    const int n = n0 + i % kHalf;
                    bias[i] = n < e.N ? load_as_float(e.bias, (size_t)(i / kHalf) * e.N + n, e.bias_type) : 0.0f;
                }
                __syncwarp();
            }
            // whole chunks move in 16-byte pieces, the residual's next one ahead
            auto whole = [&](int c) { return e.vec && m + 32 <= e.M && n0 + c + kChunk <= e.N; };
            const size_t at0 = (size_t)(m + row) * e.ldo + n0 + piece * (16 / SZ);
            const size_t rt0 = (size_t)(m + row) * e.ldr + n0 + piece * (16 / SZ);
            uint4 next[4];
            auto fetch = [&](int c) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    next[i] = *reinterpret_cast<const uint4*>(static_cast<const V*>(e.residual) + rt0 + (size_t)(8 * i) * e.ldr + c);
            };
            if (e.residual) {  // the first chunk's before the wait for the products
                if (whole(0)) fetch(0);
                else move_values<V, false>(stage, const_cast<void*>(e.residual), e.ldr, m, n0, e.M, e.N, lane);
            }
            // [0, kHalf) of the outputs (the gate's), then the up projection's
            float sum[CHAINED ? BN / 2 : 1];
            auto ready = [&] {
                if (!mbar_wait_bounded(&acc_full[b], phase)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                tc::fence_after();
                return tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * C::kIssuers * BN + half * kHalf);
            };
            auto release = [&] {
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::peer_arrive(tc::peer_addr(smem_u32(&acc_empty[b]), 0));
                if (++b == 2) b = 0, phase ^= 1u;
            };
            if constexpr (CHAINED) {
#pragma unroll
                for (int i = 0; i < BN / 2; ++i) sum[i] = 0.0f;
#pragma unroll 1
                for (int k0 = 0; k0 < nk; k0 += k0 == 0 ? chain0 : chain) {
                    const uint32_t acc = ready();
                    if (!ok) break;
#pragma unroll
                    for (int g = 0; g < BN / 2; g += 16) {
                        uint32_t v[C::kIssuers][16];
#pragma unroll
                        for (int x = 0; x < C::kIssuers; ++x)
                            tc::tmem_load16(acc + (uint32_t)(x * BN + (g < kHalf ? g : kOut + g - kHalf)), v[x]);
                        tc::tmem_wait();
#pragma unroll
                        for (int x = 0; x < C::kIssuers; ++x) {
                            tc::tmem_ready(v[x]);
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[g + i] += __uint_as_float(v[x][i]);
                        }
                    }
                    release();
                }
            }
            const uint32_t acc = CHAINED ? 0u : ready();
#pragma unroll 1  // the activations' code once
            for (int c = 0; c < kHalf; c += kChunk) {
                if (!ok) break;
                if (n0 + c >= e.N || m >= e.M) break;
                const bool pieces = whole(c);
                if (e.residual) {
                    if (pieces) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(staged(stage, row + 8 * i, piece)) = next[i];
                        if (c + kChunk < kHalf && whole(c + kChunk)) fetch(c + kChunk);
                    } else if (c > 0) {
                        move_values<V, false>(stage, const_cast<void*>(e.residual), e.ldr, m, n0 + c, e.M, e.N, lane);
                    }
                    __syncwarp();
                }
                float f[kChunk], up[kChunk];
                if constexpr (CHAINED) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        f[i] = sum[i];
                        up[i] = GATED ? sum[kHalf + i] : 0.0f;
                    }
                    // registers have no index: the next chunk's move up
#pragma unroll
                    for (int i = 0; i < BN / 2 - kChunk; ++i) sum[i] = sum[i + kChunk];
                } else {
#pragma unroll
                    for (int h = 0; h < kChunk; h += 16) {
                        uint32_t v[C::kIssuers][16], u[C::kIssuers][16];
#pragma unroll
                        for (int x = 0; x < C::kIssuers; ++x) {
                            tc::tmem_load16(acc + (uint32_t)(x * BN + c + h), v[x]);
                            if (GATED) tc::tmem_load16(acc + (uint32_t)(x * BN + kOut + c + h), u[x]);
                        }
                        tc::tmem_wait();
#pragma unroll
                        for (int x = 0; x < C::kIssuers; ++x) {
                            tc::tmem_ready(v[x]);
                            if (GATED) tc::tmem_ready(u[x]);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            f[h + i] = __uint_as_float(v[0][i]);
                            up[h + i] = GATED ? __uint_as_float(u[0][i]) : 0.0f;
                            if constexpr (C::kIssuers == 2) {
                                f[h + i] += __uint_as_float(v[1][i]);
                                if (GATED) up[h + i] += __uint_as_float(u[1][i]);
                            }
                        }
                    }
                }
                if (e.bias) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) f[i] += bias[c + i];
                }
                activate<kChunk, SZ == 4>(f, e.act);
                if (GATED) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) f[i] *= up[i] + (e.bias ? bias[kHalf + c + i] : 0.0f);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    constexpr int kPer = 16 / SZ;
                    uint4* p = reinterpret_cast<uint4*>(staged(stage, lane, j));
                    if (e.residual) {
                        const uint4 o = *p;
                        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (SZ == 4) {
                                f[j * kPer + i] += __uint_as_float(w[i]);
                            } else {
                                const float2 r = unpack2(w[i], e.out_type);
                                f[j * kPer + 2 * i] += r.x;
                                f[j * kPer + 2 * i + 1] += r.y;
                            }
                        }
                    }
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (SZ == 4) w[i] = __float_as_uint(f[j * kPer + i]);
                        else w[i] = pack2(f[j * kPer + 2 * i], f[j * kPer + 2 * i + 1], e.out_type);
                    }
                    *p = make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
                if (pieces) {
                    uint4 o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const uint4*>(staged(stage, row + 8 * i, piece));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(static_cast<V*>(e.out) + at0 + (size_t)(8 * i) * e.ldo + c) = o[i];
                } else {
                    move_values<V, true>(stage, e.out, e.ldo, m, n0 + c, e.M, e.N, lane);
                }
                __syncwarp();
            }
            if (!CHAINED) release();
        }
    }
    if (!ok && lane == 0) set_status(&g_status, MPE_STATUS_WAIT_TIMEOUT);
    tc::fence_before();
    __syncwarp();
    tc::cluster_sync();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_free_pair(tbase, C::kCols);
    }
}

typedef CUresult (*TensorMapEncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                         const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                         CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                         CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once through the runtime.
TensorMapEncodeTiled encoder() {
    static const TensorMapEncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<TensorMapEncodeTiled>(p);
    }();
    return fn;
}

// [rows x K] 16-bit values with pitch ld, read as boxes of box_rows x 64.
bool encode(CUtensorMap* map, const void* base, int type, int64_t rows, int64_t K, int64_t ld, int box_rows) {
    TensorMapEncodeTiled enc = encoder();
    if (!enc) return false;
    if (rows == 1) ld = (K + 7) / 8 * 8;  // a single row's pitch is not used, but has to be valid
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)kKStep, (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return enc(map, type == MPE_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
               const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, int S, bool GATED>
cudaError_t launch_narrow(const mpe_linear_args& p, const Epilogue& e, cudaStream_t st) {
    using C = Narrow<NT>;
    constexpr int kOut = GATED ? kRows / 2 : kRows;
    alignas(64) CUtensorMap mw, mx;
    const int64_t wrows = GATED ? 2 * (int64_t)p.N : p.N;
    if (!encode(&mw, p.w, p.type, wrows, p.K, p.ldw, kOut) || !encode(&mx, p.x, p.type, p.M, p.K, p.ldx, NT))
        return cudaErrorInvalidValue;
    cudaError_t err = cudaFuncSetAttribute(k_narrow<NT, S, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N + kOut - 1) / kOut * S), (unsigned)((p.M + NT - 1) / NT));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)S, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const int nk = (p.K + kKStep - 1) / kKStep;
    return cudaLaunchKernelEx(&cfg, k_narrow<NT, S, GATED>, mw, mx, e, nk,
                              first_chain(type_bytes(p.out_type)) / kKStep, tc::instr_desc(kRows, NT, p.type == MPE_TYPE_BF16));
}

template <int NT, bool GATED>
cudaError_t launch_narrow_split(const mpe_linear_args& p, const Epilogue& e, int split, cudaStream_t st) {
    switch (split) {
        case 1: return launch_narrow<NT, 1, GATED>(p, e, st);
        case 2: return launch_narrow<NT, 2, GATED>(p, e, st);
        case 4: return launch_narrow<NT, 4, GATED>(p, e, st);
        default: return launch_narrow<NT, 8, GATED>(p, e, st);
    }
}

template <bool GATED>
cudaError_t launch_narrow_for(const mpe_linear_args& p, const Epilogue& e, int nt, int split, cudaStream_t st) {
    switch (nt) {
        case 16: return launch_narrow_split<16, GATED>(p, e, split, st);
        case 32: return launch_narrow_split<32, GATED>(p, e, split, st);
        case 64: return launch_narrow_split<64, GATED>(p, e, split, st);
        default: return launch_narrow_split<128, GATED>(p, e, split, st);
    }
}

template <int BN, bool GATED, int SZ, bool CHAINED>
cudaError_t launch_wide(const mpe_linear_args& p, const Epilogue& e, int sms, cudaStream_t st) {
    using C = Wide<BN, CHAINED>;
    alignas(64) CUtensorMap mx, mw;
    const int64_t wrows = GATED ? 2 * (int64_t)p.N : p.N;
    if (!encode(&mx, p.x, p.type, p.M, p.K, p.ldx, 128) || !encode(&mw, p.w, p.type, wrows, p.K, p.ldw, BN / 2))
        return cudaErrorInvalidValue;
    cudaError_t err = cudaFuncSetAttribute(k_wide<BN, GATED, SZ, CHAINED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (err != cudaSuccess) return err;
    if constexpr (CHAINED) {
        // a block that starts with fewer registers than it shares out would wait for ever
        static std::atomic<bool> enough{false};
        if (!enough) {
            cudaFuncAttributes a;
            err = cudaFuncGetAttributes(&a, k_wide<BN, GATED, SZ, CHAINED>);
            if (err != cudaSuccess) return err;
            if (a.numRegs != C::kRegs) return cudaErrorLaunchOutOfResources;
            enough = true;
        }
    }
    constexpr int kOut = GATED ? BN / 2 : BN;
    const Tiles g{(p.M + kTileM - 1) / kTileM, (p.N + kOut - 1) / kOut};
    const int64_t tiles = (int64_t)g.m * g.n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)(tiles < sms / 2 ? tiles : sms / 2));
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {2, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // steps for every issuer alike: a box past K reads as zeros
    const int nk = (p.K + kKStep - 1) / kKStep, steps = (nk + C::kIssuers - 1) / C::kIssuers * C::kIssuers;
    return cudaLaunchKernelEx(&cfg, k_wide<BN, GATED, SZ, CHAINED>, mx, mw, e, g, steps,
                              tc::instr_desc(kTileM, BN, p.type == MPE_TYPE_BF16));
}

template <int BN, int SZ>
cudaError_t launch_wide_as(const mpe_linear_args& p, const Epilogue& e, int sms, cudaStream_t st) {
    if (p.K > Wide<BN, true>::kIssuers * first_chain(SZ))
        return p.gated ? launch_wide<BN, true, SZ, true>(p, e, sms, st) : launch_wide<BN, false, SZ, true>(p, e, sms, st);
    return p.gated ? launch_wide<BN, true, SZ, false>(p, e, sms, st) : launch_wide<BN, false, SZ, false>(p, e, sms, st);
}

cudaError_t launch_wide_for(const mpe_linear_args& p, const Epilogue& e, int bn, int sms, cudaStream_t st) {
    // float32: the narrower tile, whose results' chunks are as many
    if (p.out_type == MPE_TYPE_F32) return launch_wide_as<128, 4>(p, e, sms, st);
    return bn == 128 ? launch_wide_as<128, 2>(p, e, sms, st) : launch_wide_as<256, 2>(p, e, sms, st);
}

// The kernel for a product: k_wide<tile> (wide) or k_narrow<tile, split>.
struct Choice {
    bool wide;
    int tile, split;
};

// The form with the least estimated time, in us, from times measured on B200 over
// M 1 .. 8192, N 16 .. 14336, K 64 .. 14336 (of 60 products at random the form taken
// is within 10% of the best of all forms for 56, at worst 1.3 times it):
//   k_narrow<NT>  starts and ends in 3.3 + 0.025 NT (one tile, K = 2048, split 8: 3.8
//                 with NT 16, 4.1, 4.9 and 6.9 with 128); a step takes a CTA 0.24, or
//                 what an SM takes in at 105 GB/s where it has several CTAs (NT
//                 tokens x 2048 x 2048, split 1, 2, 4: 11.9, 8.3, 6.4 with NT 16,
//                 14.6, 11.3, 9.6 with 128); tiles of tokens that read the same rows
//                 of w at once get in each other's way, 0.003 a tile and step (786 x
//                 48 x 1056: 9.4 with NT 16, 6.9 with 32, 6.3 with 64); rows that do
//                 not start at 128 bytes take in two lines instead of one (333 x
//                 4096 x 2048, NT 64: 17; x 2040: 26); an SM holds three CTAs
//                 with NT 16, two with 32 and 64, one with 128, and a second round
//                 starts and ends again, mostly hidden (512 x 7168 x 2048: 33 with NT
//                 64 against 16.9 for k_wide<256>)
//   k_wide<BN>    starts and ends in 7 (BN 256: 8); a step of a pair of CTAs takes
//                 0.28 with 256, 0.17 with 128, 0.21 in a second round and later; a
//                 round's epilogue hides a short round (4.0, 2.2); rows that do not
//                 start at 128 bytes cost half as much again (333 x 4096 x 2048 and
//                 2040 with 128: 13.5, 15.5)
//                 (1024 x 2048 x 2048: 12.0 with 128, 16.0 with 256, 18 for
//                 k_narrow<64>; 512 x 2048 x 7168: 26, 39, and 28.5 for
//                 k_narrow<128> with split 2; 2048 x 2048 x 768: 11.1, 10.6)
// and all of them the time of memory at 6 TB/s, which hides most of the steps (or
// is hidden by them).
Choice choose(const mpe_linear_args& p, int sms) {
    const int nk = (p.K + kKStep - 1) / kKStep;
    const int per = p.gated ? kRows / 2 : kRows;
    const double wrows = p.gated ? 2.0 * p.N : p.N;
    const double memory =
        (2.0 * p.K * (p.M + wrows) + (p.residual ? 2.0 : 1.0) * type_bytes(p.out_type) * p.M * p.N) / 6e6;
    auto both = [&](double steps) { return (steps > memory ? steps : memory) + 0.25 * (steps > memory ? memory : steps); };
    // rows that start at 128 bytes
    const bool lines = (p.N == 1 || p.ldw % 64 == 0) && (p.M == 1 || p.ldx % 64 == 0) && aligned(p.w, 128) && aligned(p.x, 128);
    Choice best{true, 256, 1};
    double least = 1e30;
    auto offer = [&](const Choice& c, double us) {
        if (us < least) best = c, least = us;
    };
    for (int bn = 128; bn <= (p.out_type == MPE_TYPE_F32 ? 128 : 256); bn += 128) {
        const int out = p.gated ? bn / 2 : bn;
        const double tiles = (double)((p.M + kTileM - 1) / kTileM) * ((p.N + out - 1) / out);
        const double rounds = (double)(int64_t)((tiles + sms / 2 - 1) / (sms / 2));
        const double steps = nk * (bn == 256 ? 0.28 : rounds > 1 ? 0.21 : 0.17) * (lines ? 1.0 : 1.5), epilogue = bn == 256 ? 4.0 : 2.2;
        offer({true, bn, 1}, (bn == 256 ? 8.0 : 7.0) + both(steps + (rounds - 1) * (steps > epilogue ? steps : epilogue)));
    }
    const int64_t ntiles = (p.N + per - 1) / per;
    for (int nt = 16; nt <= 128 && nt / 2 < p.M + 8; nt *= 2) {  // the next above M, too
        const int64_t mtiles = (p.M + nt - 1) / nt;
        if (mtiles > 65535) continue;  // the grid's y
        const double fixed = 3.3 + 0.025 * nt + 0.003 * mtiles * nk, ingest = (kRows + nt) * 128 / 105e3;
        for (int s = 1; s <= 8 && (s == 1 || nk >= 2 * s); s *= 2) {
            const double ctas = (double)ntiles * mtiles * s, slots = nt == 128 ? sms : nt == 16 ? 3 * sms : 2 * sms;
            if (ntiles * s > INT32_MAX) continue;  // the grid's x
            const double rounds = (double)(int64_t)((ctas + slots - 1) / slots);
            const double there = (ctas < slots ? ctas : slots) / sms;  // CTAs an SM
            const double in = there * ingest * (lines ? 1.0 : 1.9), step = in > 0.24 ? in : 0.24;
            offer({false, nt, s}, fixed + 0.7 * fixed * (rounds - 1) + both(rounds * ((nk + s - 1) / s) * step));
        }
    }
    return best;
}

}  // namespace
}  // namespace mpe

using namespace mpe;

extern "C" int mpe_linear(const mpe_linear_args* p, void* stream) {
    constexpr const char* who = "mpe_linear";
    if (!p) return report_global_error(MPE_ERR_INVALID, "mpe_linear: null args");
    constexpr int64_t kMaxDim = 1 << 30, kMaxLd = (int64_t)1 << 38;
    if (p->M < 0 || p->N < 1 || p->K < 1 || p->M > kMaxDim || p->N > kMaxDim || p->K > kMaxDim)
        return report_global_errorf(MPE_ERR_INVALID, "%s: M=%d N=%d K=%d", who, p->M, p->N, p->K);
    if (p->type != MPE_TYPE_BF16 && p->type != MPE_TYPE_F16)
        return report_global_errorf(MPE_ERR_INVALID, "%s: type %d is not bf16 or f16", who, p->type);
    if (p->out_type != p->type && p->out_type != MPE_TYPE_F32)
        return report_global_errorf(MPE_ERR_INVALID, "%s: out_type %d for type %d", who, p->out_type, p->type);
    if (p->bias && p->bias_type != p->type && p->bias_type != MPE_TYPE_F32)
        return report_global_errorf(MPE_ERR_INVALID, "%s: bias_type %d for type %d", who, p->bias_type, p->type);
    if (p->act < MPE_ACT_NONE || p->act > MPE_ACT_GELU_TANH)
        return report_global_errorf(MPE_ERR_INVALID, "%s: bad act %d", who, p->act);
    if (p->M == 0) return MPE_OK;
    if (!p->x || !p->w || !p->out) return report_global_errorf(MPE_ERR_INVALID, "%s: null x, w or out", who);
    const int64_t wrows = p->gated ? 2 * (int64_t)p->N : p->N;
    auto bad_ld = [](int64_t rows, int64_t ld, int64_t cols, int64_t step) {
        return rows > 1 && (ld < cols || ld >= kMaxLd || ld % step);
    };
    if (bad_ld(p->M, p->ldx, p->K, 8) || bad_ld(wrows, p->ldw, p->K, 8))
        return report_global_errorf(MPE_ERR_INVALID, "%s: ldx=%lld ldw=%lld for K=%d (multiples of 8)", who,
                                    (long long)p->ldx, (long long)p->ldw, p->K);
    if (bad_ld(p->M, p->ldo, p->N, 1) || (p->residual && bad_ld(p->M, p->ldr, p->N, 1)))
        return report_global_errorf(MPE_ERR_INVALID, "%s: ldo=%lld ldr=%lld for N=%d", who, (long long)p->ldo,
                                    (long long)p->ldr, p->N);
    const int osz = type_bytes(p->out_type);
    if (!aligned(p->x, 16) || !aligned(p->w, 16))
        return report_global_errorf(MPE_ERR_INVALID, "%s: x or w not 16-byte aligned", who);
    if (!aligned(p->out, osz) || !aligned(p->residual, osz) ||
        (p->bias && !aligned(p->bias, type_bytes(p->bias_type))))
        return report_global_errorf(MPE_ERR_INVALID, "%s: out, residual or bias not aligned to its type", who);
    const Block out(p->out, p->M, p->N, p->ldo, osz);
    if (overlap(out, Block(p->x, p->M, p->K, p->ldx, 2)) || overlap(out, Block(p->w, wrows, p->K, p->ldw, 2)) ||
        (p->bias && overlap(out, Block(p->bias, 1, wrows, wrows, type_bytes(p->bias_type)))))
        return report_global_errorf(MPE_ERR_INVALID, "%s: out overlaps x, w or bias", who);
    if (p->residual && !(p->residual == p->out && (p->M == 1 || p->ldr == p->ldo)) &&
        overlap(out, Block(p->residual, p->M, p->N, p->ldr, osz)))
        return report_global_errorf(MPE_ERR_INVALID, "%s: out overlaps residual without being it", who);
    const int sms = current_sm_count();
    if (sms <= 0) return report_global_errorf(MPE_ERR_CUDA, "%s: no current device", who);
    const Choice how = choose(*p, sms);
    // rows start where runs of 16 bytes (narrow: of 4 values) do
    const int run = how.wide ? 16 : 4 * osz;
    auto runs = [&](const void* base, int64_t ld) { return aligned(base, run) && (p->M == 1 || ld * osz % run == 0); };
    const int vec = runs(p->out, p->ldo) && (!p->residual || runs(p->residual, p->ldr));
    const Epilogue e{p->bias, p->residual, p->out, p->ldr, p->ldo, p->M, p->N, p->bias_type, p->out_type, p->act, vec};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = how.wide   ? launch_wide_for(*p, e, how.tile, sms, st)
                            : p->gated ? launch_narrow_for<true>(*p, e, how.tile, how.split, st)
                                       : launch_narrow_for<false>(*p, e, how.tile, how.split, st);
    if (err != cudaSuccess) {
        cudaGetLastError();  // reported here, not left for the next call
        return report_global_errorf(MPE_ERR_CUDA, "%s: %s", who, cudaGetErrorString(err));
    }
    return MPE_OK;
}

extern "C" int mpe_global_status(uint32_t* status_out, int32_t clear) {
    constexpr const char* who = "mpe_global_status";
    if (!status_out) return report_global_error(MPE_ERR_INVALID, "mpe_global_status: null argument");
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(status_out, g_status, sizeof(uint32_t));
    const uint32_t zero = 0;
    if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(zero));
    if (e != cudaSuccess) return report_global_errorf(MPE_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return MPE_OK;
}
