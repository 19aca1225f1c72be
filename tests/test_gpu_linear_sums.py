"""mpe_linear's sums over K on values whose products do not fit float32 exactly, against float64.

The tensor cores cut what they add to an accumulator: an instruction of 16 inputs loses less than one unit
of the accumulator's last place, 2^-23 of it, always towards zero. An accumulator takes 512 inputs (float32
results; 32 instructions) or 1024, the first time up to 2048 (16-bit results; 128), then it starts again and its
sum is added up in float32, rounding to nearest: 2^-24 an addition, at most one for every such run of inputs, one
for every two issuers' and one for every rank's. So a sum of terms of one sign is off by at most

    n 2^-23 + (K / inputs + 10) 2^-24,   n = 32 and inputs = 512, or n = 128 and inputs = 1024,

of itself, and one of both signs by that much of the sum of magnitudes. A 16-bit result is rounded once: half a
step of the result's binade."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def mpe():
    import mixed_precision_expert_b200 as m
    m.lib()
    return m


def bound(K, out):
    n, inputs = (32, 512) if out == "f32" else (128, 1024)
    return n * 2.0 ** -23 + (K / inputs + 10) * 2.0 ** -24


def half_step(v, out):
    """Half the distance of out's values in v's binade (v float64, normal in out)."""
    return torch.exp2(torch.floor(torch.log2(v.abs()))) * (torch.finfo(DT[out]).eps / 2)


def operands(M, N, K, dtype, seed, signed=False):
    """Rows at multiples of 8 values; magnitudes in [1/2, 1) / sqrt(K / 256), so that a sum is near 144."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for rows in (M, N):
        t = torch.zeros(rows, (K + 7) // 8 * 8, dtype=DT[dtype], device="cuda")
        for r0 in range(0, rows, 64):
            r1 = min(rows, r0 + 64)
            v = torch.rand(r1 - r0, K, generator=g, device="cuda") * 0.5 + 0.5
            if signed:
                v *= torch.randint(0, 2, v.shape, generator=g, device="cuda") * 2 - 1
            t[r0:r1, :K] = (v * (256 / K) ** 0.5).to(DT[dtype])
        out.append(t[:, :K])
    return out


def product64(x, w):
    """x w^T in float64, a slice of K at a time."""
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for k in range(0, x.shape[1], 1 << 18):
        total += x[:, k:k + (1 << 18)].double() @ w[:, k:k + (1 << 18)].double().t()
    return total


# both kernels, one and several tiles of tokens, one run of inputs and many, a last run of one step
SIZES = [(1, 96, 7168), (8, 130, 14336), (64, 128, 7168), (128, 260, 40000), (300, 512, 14336), (1024, 2048, 1040),
         (1024, 2048, 2056), (2048, 1024, 40000), (700, 3000, 7170), (4, 64, 1 << 21)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
def test_sums_of_one_sign(mpe, M, N, K, dtype, out):
    x, w = operands(M, N, K, dtype, 3)
    ref = product64(x, w)
    got = mpe.linear(x, w, out_dtype=DT[out]).double()
    tol = ref * bound(K, out)
    if out != "f32":
        tol = tol + half_step(ref + tol, out)
    off = (got - ref).abs()
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / ref).max()))


@pytest.mark.parametrize("M,N,K", [(2, 200, 20000), (200, 384, 14336), (1500, 1024, 9000)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gated_sums(mpe, M, N, K, out):
    """Both factors keep their bound; a product and its rounding."""
    x, w = operands(M, 2 * N, K, "bf16", 5)
    ref = product64(x, w[:N]) * product64(x, w[N:])
    got = mpe.linear(x, w, gated=True, out_dtype=DT[out]).double()
    tol = ref * (2.01 * bound(K, out) + 2.0 ** -24)
    if out != "f32":
        tol = tol + half_step(ref + tol, out)
    off = (got - ref).abs()
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / ref).max()))


@pytest.mark.parametrize("M,N,K", [(3, 300, 30000), (900, 1000, 14336)])
def test_sums_of_both_signs(mpe, M, N, K):
    x, w = operands(M, N, K, "bf16", 7, signed=True)
    off = (mpe.linear(x, w, out_dtype=torch.float32).double() - product64(x, w)).abs()
    assert (off <= product64(x.abs(), w.abs()) * bound(K, "f32")).all()


def test_long_sums_with_every_part_of_the_epilogue(mpe):
    M, N, K = 333, 1027, 9000
    g = torch.Generator(device="cuda").manual_seed(9)
    x, w = operands(M, N, K, "f16", 11)
    b = torch.randn(N, generator=g, device="cuda").half()
    r = torch.randn(M, N, generator=g, device="cuda").half()
    ref = product64(x, w) + b.double() + r.double()
    tol = product64(x, w) * bound(K, "f16") + 2 * (ref.abs() + 8) * 2.0 ** -24  # two additions in float32
    off = (mpe.linear(x, w, bias=b, act=mpe.ACT_RELU, residual=r).double() - ref).abs()
    assert (off <= tol + half_step(ref + tol, "f16")).all()
