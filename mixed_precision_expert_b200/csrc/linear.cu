// out = act(x w^T + bias) + residual and its gated form (mpe_linear).
#include <cstdio>

#include "internal.h"
#include "opcheck.h"

namespace mpe {
namespace {

// Sticky status of the current device's context-free calls.
__device__ uint32_t g_status;

struct LinearArgs {
    const void *x, *w, *bias, *residual;
    void* out;
    int64_t ldx, ldw, ldr, ldo;
    int M, N, K, type, bias_type, out_type, act, gated;
};

__device__ __forceinline__ float load_as_float(const void* p, size_t i, int type) {
    if (type == MPE_TYPE_F32) return static_cast<const float*>(p)[i];
    if (type == MPE_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case MPE_ACT_RELU: return v < 0.0f ? 0.0f : v;
        case MPE_ACT_SILU: return v / (1.0f + expf(-v));
        case MPE_ACT_GELU: return 0.5f * v * erfcf(-0.70710678f * v);
        case MPE_ACT_GELU_TANH: return v / (1.0f + expf(-1.59576912f * (v + 0.044715f * v * v * v)));
        default: return v;
    }
}

// One 64 x 64 tile of outputs a block, 16 inputs a step, 4 x 4 outputs a thread.
__global__ void __launch_bounds__(256) k_linear(const LinearArgs a) {
    __shared__ float xs[16][65], ws[2][16][65];
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
    float acc[2][4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i / 16, c = i % 16, k = k0 + c;
            xs[c][r] = m0 + r < a.M && k < a.K ? load_as_float(a.x, (size_t)(m0 + r) * a.ldx + k, a.type) : 0.0f;
            for (int h = 0; h <= a.gated; ++h)
                ws[h][c][r] = n0 + r < a.N && k < a.K
                                  ? load_as_float(a.w, ((size_t)h * a.N + n0 + r) * a.ldw + k, a.type)
                                  : 0.0f;
        }
        __syncthreads();
        for (int c = 0; c < 16; ++c)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    acc[0][i][j] += xs[c][tm + i] * ws[0][c][tn + j];
                    if (a.gated) acc[1][i][j] += xs[c][tm + i] * ws[1][c][tn + j];
                }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + tm + i, n = n0 + tn + j;
            if (m >= a.M || n >= a.N) continue;
            float v = acc[0][i][j], u = acc[1][i][j];
            if (a.bias) {
                v += load_as_float(a.bias, n, a.bias_type);
                if (a.gated) u += load_as_float(a.bias, (size_t)a.N + n, a.bias_type);
            }
            v = activate(v, a.act);
            if (a.gated) v *= u;
            if (a.residual) v += load_as_float(a.residual, (size_t)m * a.ldr + n, a.out_type);
            const size_t o = (size_t)m * a.ldo + n;
            if (a.out_type == MPE_TYPE_F32) static_cast<float*>(a.out)[o] = v;
            else if (a.out_type == MPE_TYPE_BF16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
            else static_cast<__half*>(a.out)[o] = __float2half_rn(v);
        }
}

// rows of `cols` values of sz bytes, ld values apart, as a set of bytes
struct Block {
    uintptr_t base;
    int64_t pitch, width, rows;
    Block(const void* p, int64_t r, int64_t cols, int64_t ld, int sz)
        : base(reinterpret_cast<uintptr_t>(p)), pitch(r > 1 ? ld * sz : cols * sz), width(cols * sz), rows(r) {}
    uintptr_t end() const { return base + (uintptr_t)((rows - 1) * pitch + width); }
};

// Whether two blocks share a byte. Blocks of one pitch whose spans interleave
// (columns of one buffer) share none when their columns do not meet; blocks of
// different pitches count as overlapping when their spans do.
bool overlap(const Block& p, const Block& q) {
    if (p.end() <= q.base || q.end() <= p.base) return false;
    if (p.rows > 1 && q.rows > 1 && p.pitch == q.pitch) {
        // where q's rows start in p's
        const int64_t at = q.base >= p.base ? (int64_t)(q.base - p.base) % p.pitch
                                            : (p.pitch - (int64_t)(p.base - q.base) % p.pitch) % p.pitch;
        return at < p.width || at + q.width > p.pitch;
    }
    return true;
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
    LinearArgs a{p->x,   p->w,   p->bias, p->residual, p->out,       p->ldx,      p->ldw, p->ldr,      p->ldo,
                 p->M,   p->N,   p->K,    p->type,     p->bias_type, p->out_type, p->act, p->gated != 0};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    k_linear<<<dim3((p->N + 63) / 64, (p->M + 63) / 64), 256, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return report_global_errorf(MPE_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
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
