"""mpe_linear against the float64 oracle.

Inputs are small multiples of powers of two, so that every product and every
partial sum is a multiple of 2^-6 below 2^18 and exact in float32 in any order:
without an activation the result is the exact value rounded once, and a product
that is missing, doubled or misplaced shows. An activation of the exact v is off by
at most |v| 2^-19: a sigmoid by 2^-22 and the rounding of its argument, the normal
distribution function by 7.5e-8, both with a reciprocal and a product of 1 ulp, times
v. Its result is rounded once more."""
import numpy as np
import pytest
import torch

from oracle import linear as oln

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def mpe():
    import mixed_precision_expert_b200 as m
    m.lib()
    return m


def grid(rows, cols, step, dtype, seed, pad=None):
    """Multiples of step in [-4 step, 4 step], rows at multiples of 8 values, NaN in the padding."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pitch = (cols + 7) // 8 * 8 + (8 if pad is None else pad)
    full = torch.full((rows, pitch), float("nan"), dtype=DT[dtype], device="cuda")
    full[:, :cols] = (torch.randint(-4, 5, (rows, cols), generator=g, device="cuda") * step).to(DT[dtype])
    return full[:, :cols]


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def rounded(ref, dtype):
    return torch.from_numpy(ref).to(DT[dtype]) if dtype != "f32" else torch.from_numpy(ref).float()


def check(mpe, M, N, K, dtype="bf16", out="bf16", act="none", gated=False, bias=None, residual=False, step=0.125,
          seed=0, pad=None, inplace=False):
    rows = 2 * N if gated else N
    x = grid(M, K, step, dtype, 11 + seed, pad)
    w = grid(rows, K, step, dtype, 23 + seed, pad)
    b = None if bias is None else grid(1, rows, 0.25, bias, 37 + seed)[0].contiguous()
    r = grid(M, N, 0.5, out, 41 + seed, 1) if residual else None
    # the frame around out, which has to stay as it is
    frame = torch.full((M + 2, N + 5), -77.0, dtype=DT[out], device="cuda")
    o = frame[1:M + 1, 2:N + 2]
    if inplace:
        o.copy_(r)
    got = mpe.linear(x, w, bias=b, act=getattr(mpe, "ACT_" + act.upper()), gated=gated,
                     residual=o if inplace else r, out=o)
    assert got is o
    rest = frame.clone()
    rest[1:M + 1, 2:N + 2] = -77.0
    assert (rest == -77.0).all(), "wrote outside out"
    ref = oln.linear(f64(x), f64(w), f64(b), act, gated, f64(r))
    if act in ("none", "relu"):
        want = rounded(ref, out)
        assert torch.equal(got.cpu(), want), (got.cpu().double() - want.double()).abs().max()
        return
    pre = oln.preactivation(f64(x), f64(w), f64(b))
    v, up = (np.abs(pre[:, :N]), np.abs(pre[:, N:])) if gated else (np.abs(pre), 1.0)
    half = torch.finfo(DT[out]).eps / 2
    early = v * up * 2.0 ** -19 + np.abs(ref) * 2.0 ** -23 + (0 if r is None else np.abs(f64(r)) * 2.0 ** -23)
    tol = early + (np.abs(ref) + early) * half + 2.0 ** -25  # f16: half a step of its smallest values
    assert (np.abs(f64(got) - ref) <= tol).all(), (np.abs(f64(got) - ref) - tol).max()


@pytest.mark.parametrize("M", [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 96, 127, 128, 129, 200, 256, 257, 300])
def test_tokens(mpe, M):
    check(mpe, M, 136, 200)
    check(mpe, M, 131, 128, "f16", "f32", bias="f16", residual=True)
    check(mpe, M, 130, 320, gated=True)


@pytest.mark.parametrize("N", [1, 2, 7, 8, 16, 63, 64, 65, 100, 127, 128, 129, 192, 255, 256, 257, 500, 1000])
def test_outputs(mpe, N):
    for M in (5, 140):
        check(mpe, M, N, 136, "bf16", "f32", residual=True)
        check(mpe, M, N, 264, "bf16", "bf16", bias="f32", gated=True)


@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 15, 16, 17, 56, 63, 64, 65, 72, 120, 127, 128, 129, 192, 255, 320, 511, 512,
                               513, 1000, 1024, 2040, 4096])
def test_inputs(mpe, K):
    for M in (1, 20, 150):
        check(mpe, M, 144, K, "f16" if K % 2 else "bf16", "f32")
        check(mpe, M, 70, K, gated=True, residual=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("gated", [False, True])
def test_epilogues(mpe, act, dtype, out, gated):
    seed = 0
    for M, N, K in ((3, 129, 24), (48, 96, 136), (130, 264, 72)):
        for bias in (None, dtype, "f32"):
            for residual in (False, True):
                seed += 1
                check(mpe, M, N, K, dtype, out, act, gated, bias, residual, seed=seed)


@pytest.mark.parametrize("M,N,K", [(512, 1024, 1024), (1000, 777, 520), (2048, 256, 512), (4096, 128, 256), (64, 7168, 2048),
                                   (1, 14336, 512), (260, 4100, 136), (300, 2048, 2040), (129, 129, 14336)])
def test_larger(mpe, M, N, K):
    check(mpe, M, N, K, residual=True)
    check(mpe, M, N // 2, K, "bf16", "bf16", bias="bf16", gated=True)
    check(mpe, M, N, K, "f16", "f32", pad=0)


def test_residual_in_place(mpe):
    for M, N in ((1, 64), (5, 200), (130, 136), (300, 513)):
        check(mpe, M, N, 128, residual=True, inplace=True)
        check(mpe, M, N, 128, "f16", "f32", bias="f16", residual=True, inplace=True)
    # the usual layout: whole rows, aligned
    x, w = grid(300, 256, 0.125, "bf16", 1, 0), grid(512, 256, 0.125, "bf16", 2, 0)
    h = grid(300, 512, 0.5, "bf16", 3, 0).contiguous()
    want = rounded(oln.linear(f64(x), f64(w), residual=f64(h)), "bf16")
    mpe.linear(x, w, residual=h, out=h)
    assert torch.equal(h.cpu(), want)


def test_columns_of_one_buffer(mpe):
    for M in (4, 200):
        buf = torch.zeros(M, 256 + 128, dtype=torch.bfloat16, device="cuda")
        buf[:, :256] = grid(M, 256, 0.125, "bf16", 5, 0)
        w = grid(128, 256, 0.125, "bf16", 6, 0)
        want = rounded(oln.linear(f64(buf[:, :256]), f64(w)), "bf16")
        mpe.linear(buf[:, :256], w, out=buf[:, 256:])
        assert torch.equal(buf[:, 256:].cpu(), want)


def test_infinities_and_nan_stay_in_their_rows(mpe):
    for M in (6, 200):
        x, w = grid(M, 128, 0.125, "bf16", 7), grid(136, 128, 0.125, "bf16", 8)
        want = rounded(oln.linear(f64(x), f64(w)), "bf16")
        x[2, 3], x[4, 5] = float("nan"), float("inf")
        w[:, 5] = 1.0
        got = mpe.linear(x, w)
        want = rounded(oln.linear(f64(x), f64(w)), "bf16")
        assert torch.isnan(got[2]).all() and torch.isposinf(got[4]).all()
        rest = [i for i in range(M) if i not in (2, 4)]
        assert torch.equal(got.cpu()[rest], want[rest])
        assert torch.isnan(mpe.linear(x, w, act=mpe.ACT_RELU)[2]).all()


def test_offsets_past_32_bits(mpe):
    """2.3e9 outputs of one product, and rows of x, w, residual and out 2^28 values apart."""
    M, N, K = 140_000, 16_384, 16
    x, w = grid(M, K, 0.125, "bf16", 61, 0), grid(N, K, 0.125, "bf16", 62, 0)
    out = mpe.linear(x, w)
    rows = torch.tensor([0, 1, 131_071, 131_072, M - 1]).cuda()
    want = rounded(oln.linear(f64(x[rows]), f64(w)), "bf16")
    assert torch.equal(out[rows].cpu(), want)
    for first in range(0, M, 20_000):  # all of it, on the device: exact products, rounded once
        part = x[first:first + 20_000].double() @ w.double().t()
        assert torch.equal(out[first:first + 20_000], part.to(torch.bfloat16))
    del part
    flat = out.view(-1)[:8 * 2 ** 28].view(8, 2 ** 28)
    for m, n, k in ((8, 8, 256), (5, 8, 100)):
        xs, ws = flat[:m, 0:k], flat[:n, 4096:4096 + k]
        xs.copy_(grid(m, k, 0.125, "bf16", 63, 0))
        ws.copy_(grid(n, k, 0.125, "bf16", 64, 0))
        o, r = flat[:m, 1 << 20:(1 << 20) + n], flat[:m, 1 << 21:(1 << 21) + n]
        r.copy_(grid(m, n, 0.5, "bf16", 65, 0))
        mpe.linear(xs, ws, residual=r, out=o)
        assert torch.equal(o.cpu(), rounded(oln.linear(f64(xs), f64(ws), residual=f64(r)), "bf16"))


def test_many_tokens_few_outputs(mpe):
    """More token tiles than a grid's y has."""
    for M, N, K in ((1_200_000, 8, 16), (1_100_000, 3, 8)):
        x, w = grid(M, K, 0.125, "bf16", 66, 0), grid(N, K, 0.125, "bf16", 67, 0)
        want = (x.double() @ w.double().t()).to(torch.bfloat16)
        assert torch.equal(mpe.linear(x, w), want)


def test_overflow_of_a_16_bit_result(mpe):
    x, w = torch.full((3, 64), 200.0).half().cuda(), torch.full((64, 64), 200.0).half().cuda()
    assert torch.isposinf(mpe.linear(x, w)).all()              # 2.56e6
    assert (mpe.linear(x, w, out_dtype=torch.float32) == 2.56e6).all()


def test_activations_far_out(mpe):
    """v of up to +-4000 through every activation: no NaN from an overflow inside."""
    x = torch.zeros(4, 64).bfloat16().cuda()
    x[:, 0] = torch.tensor([1.0, -1.0, 40.0, -40.0])
    w = torch.zeros(8, 64).bfloat16().cuda()
    w[:, 0] = torch.tensor([0.5, 1.0, 2.0, 4.0, 8.0, 20.0, 50.0, 100.0])
    v = f64(x) @ f64(w).T
    for act in ACTS:
        got = f64(mpe.linear(x, w, act=getattr(mpe, "ACT_" + act.upper()), out_dtype=torch.float32))
        assert (np.abs(got - oln.activate(v, act)) <= np.abs(v) * 2.0 ** -19 + 1e-30).all(), act


def test_on_another_stream_and_in_graphs(mpe):
    cases = []
    for M, N, K in ((4, 256, 512), (64, 128, 2048), (300, 512, 256)):
        x, w = grid(M, K, 0.125, "bf16", 9, 0), grid(N, K, 0.125, "bf16", 10, 0)
        cases.append((x, w, rounded(oln.linear(f64(x), f64(w)), "bf16").cuda()))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for x, w, want in cases:
        with torch.cuda.stream(st):
            y = x * 1.0
            got = mpe.linear(y, w)
        st.synchronize()
        assert torch.equal(got, want)
    # two graphs of the same calls, replayed on two streams at once
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        static = [torch.zeros_like(c[0]) for c in cases]
        with torch.cuda.graph(g):
            outs = [mpe.linear(s, c[1]) for s, c in zip(static, cases)]
        for s, c in zip(static, cases):
            s.copy_(c[0])
        graphs.append((g, outs))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        for o, c in zip(outs, cases):
            assert torch.equal(o, c[2])


def test_repeats_to_the_bit(mpe):
    for M, N, K in ((8, 256, 4096), (64, 128, 2048), (200, 300, 1000)):
        g = torch.Generator(device="cuda").manual_seed(3)
        x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        w = torch.randn(N, K, generator=g, device="cuda").bfloat16()
        a = mpe.linear(x, w, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(a, mpe.linear(x, w, out_dtype=torch.float32))


def test_status_stays_clear(mpe):
    assert mpe.global_status(clear=True) == 0
