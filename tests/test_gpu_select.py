"""mpe_select_experts and mpe_expert_importance against the float64 oracle.

Ids are equal. A float32 weight is off by at most: the exponential's 2 ulp (4
units of 2^-24) and the rounding of its argument, l - max (one unit of its
size), in the numerator and in the mean of the denominator's terms; up to 31 + 5
roundings of the sum; reciprocal, products, scale: 8 units. An importance has the fast
exponential's 2 + 1.2 d ulp for a score of e^-d (so 4 + 3.4 d units in the numerator and,
with a mean d below 7, 28 in the denominator), 36 roundings of the sum, 8 of the division
and product, and 256 + 17 of partial sums and its own."""
import numpy as np
import pytest
import torch

from oracle import select as osel

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = float("inf")


@pytest.fixture(scope="module")
def mpe():
    import mixed_precision_expert_b200 as m
    m.lib()
    return m


def importance_tol(l, ref):
    fin = l[np.isfinite(l)]
    return ref * (3.4 * (fin.max() - fin.min()) + 80 + 256 + 17) * U


def weight_tol(l, ref):
    fin = np.where(np.isfinite(l), l, 0.0)
    spread = fin.max(axis=1) - fin.min(axis=1)
    return np.abs(ref) * ((2 * spread + 60) * U)[:, None] + 2.0 ** -126


def check(mpe, l, k, dtype="f32", got=None, **kw):
    """select_experts on l (a torch tensor of any of the types, on the GPU) against the oracle."""
    names = {"score": {"softmax": mpe.SCORE_SOFTMAX, "sigmoid": mpe.SCORE_SIGMOID},
             "group_score": {"max": mpe.GROUP_MAX, "top2": mpe.GROUP_TOP2}}
    bias = kw.get("bias")
    call = {n: names[n][v] if n in names else v for n, v in kw.items()}
    ids, w = mpe.select_experts(l, k, **call)
    ref_kw = dict(kw, bias=None if bias is None else bias.double().cpu().numpy())
    l64 = l.double().cpu().numpy()
    rid, rw = osel.select_experts(l64, k, **ref_kw)
    ids, w = ids.cpu().numpy(), w.double().cpu().numpy()
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:4]
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert (np.abs(w - rw)[ok] <= weight_tol(l64, rw)[ok]).all()


def logits(T, E, dtype="f32", seed=0, sigma=1.5):
    g = torch.Generator().manual_seed(seed * 1000003 + T * 1031 + E)
    return (torch.randn(T, E, generator=g) * sigma).to(DT[dtype]).cuda()


@pytest.mark.parametrize("E", [1, 2, 8, 31, 32, 33, 60, 64, 100, 128, 160, 255, 256, 257, 384, 512, 513, 1000, 1024])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_expert_counts(mpe, E, dtype):
    l = logits(9, E, dtype)
    for k in sorted({1, min(E, 8), min(E, 32)}):
        check(mpe, l, k)
        check(mpe, l, k, score="sigmoid", renormalize=False, scale=2.5)
        check(mpe, l, k, score="sigmoid", bias=torch.randn(E).cuda() * 0.1)
        check(mpe, l, k, bias=torch.randn(E).cuda() * 0.01, renormalize=False)


@pytest.mark.parametrize("T", [0, 1, 2, 3, 5, 127, 128, 129, 2368, 2369, 9001])
def test_token_counts(mpe, T):
    l = logits(T, 128, seed=2)
    ids, w = mpe.select_experts(l, 8)
    assert ids.shape == (T, 8) and w.shape == (T, 8)
    check(mpe, l, 8)


@pytest.mark.parametrize("E,G,keep,k", [(256, 8, 4, 8), (256, 8, 1, 8), (160, 8, 3, 6), (64, 32, 5, 7), (96, 3, 2, 32),
                                        (32, 32, 8, 8), (1024, 32, 4, 8), (512, 16, 15, 9), (60, 4, 2, 4), (30, 10, 7, 5),
                                        (1023, 3, 2, 8), (1020, 17, 5, 8), (14, 7, 3, 3), (31, 31, 9, 9), (672, 6, 5, 16)])
@pytest.mark.parametrize("how", ["max", "top2"])
def test_groups(mpe, E, G, keep, k, how):
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.randn(E).cuda() * 0.1):
            for dtype in ("f32", "bf16"):
                check(mpe, logits(40, E, dtype, seed=3), k, score=score, bias=bias, n_groups=G, keep_groups=keep,
                      group_score=how)


def test_ties_and_near_ties(mpe):
    # few values: most keys are equal to others, group sums too
    g = torch.Generator().manual_seed(4)
    l = torch.randint(-2, 3, (200, 96), generator=g).float().cuda()
    b = (torch.randint(0, 2, (96,), generator=g).float() * 0.25).cuda()
    for kw in ({}, dict(bias=b), dict(score="sigmoid", bias=b), dict(bias=torch.zeros(96).cuda()),
               dict(n_groups=8, keep_groups=3), dict(n_groups=8, keep_groups=3, bias=b, score="sigmoid"),
               dict(n_groups=8, keep_groups=2, group_score="max", bias=b)):
        check(mpe, l, 12, **kw)
    check(mpe, torch.zeros(3, 256).cuda(), 32, n_groups=8, keep_groups=4, score="sigmoid", bias=torch.zeros(256).cuda())
    check(mpe, torch.tensor([[0.0, -0.0, 0.0, -0.0, 1.0]]).cuda(), 4)
    # keys nearer than float32 can tell apart: neighbouring logits, and biases that undo the scores' differences
    base = torch.full((64, 128), 0.3)
    base += torch.arange(128).float()[None, torch.randperm(128, generator=g)] * 2.0 ** -24
    check(mpe, base.cuda(), 16)
    check(mpe, base.cuda(), 16, score="sigmoid", bias=torch.zeros(128).cuda())
    for score in ("softmax", "sigmoid"):
        l = torch.randn(64, 128, generator=g)
        s = torch.from_numpy(osel.scores(l.numpy(), score))
        near = (0.5 - s[0]).float()  # row 0: every key is 0.5 up to its rounding
        l[1:32] = l[0]
        check(mpe, l.cuda(), 16, score=score, bias=near.cuda())
        check(mpe, l.cuda(), 16, score=score, bias=near.cuda(), n_groups=8, keep_groups=3)


def test_orders_that_crowd_a_lane(mpe):
    """Sorted rows (the largest keys next to each other), constant rows, two levels."""
    for E in (64, 128, 256, 512, 1024):
        base = torch.arange(E).float() / 50
        rows = torch.stack([base, -base, (base * 7) % 3, torch.zeros(E), (torch.arange(E) % 2).float(),
                            (torch.arange(E) >= E - 9).float(), (torch.arange(E) < 40).float()]).cuda()
        for k in (1, 8, 16, 32):
            check(mpe, rows, k)
            check(mpe, rows, k, score="sigmoid", bias=(base * 0.001).cuda())
            check(mpe, rows, min(k, E // 4), n_groups=8, keep_groups=2, score="sigmoid", bias=torch.zeros(E).cuda())
            check(mpe, rows, min(k, E // 16), n_groups=16, keep_groups=1, group_score="max")


def test_large_biases(mpe):
    l = logits(50, 64, seed=5)
    for scale in (1e-8, 3.0, 1e4, 1e8, 1e30):
        b = torch.randn(64).cuda() * scale
        check(mpe, l, 8, score="sigmoid", bias=b)
        check(mpe, l, 8, bias=b, n_groups=8, keep_groups=4)


def test_masked_broken_and_extreme_rows(mpe):
    l = logits(12, 100, seed=6)
    l[0] = -INF                       # nothing left
    l[1, 3:] = -INF                   # three left
    l[2, 7] = float("nan")
    l[3, 9] = INF
    l[4] = float("nan")
    l[5] *= 1e4                       # scores underflow
    l[6] = -200.0                     # sigmoids below the smallest float32
    l[6, 4] = -199.0
    l[7] = 3e38
    l[8] = -3e38
    l[9, :50] = -INF
    bias = torch.randn(100).cuda() * 0.1
    bias[[3, 5]] = -INF
    check(mpe, l, 8, bias=bias)
    check(mpe, l[[0, 1, 2, 3, 9, 10]], 8, score="sigmoid", bias=bias, n_groups=10, keep_groups=4)
    bias[8] = float("nan")
    for kw in ({}, dict(n_groups=10, keep_groups=4), dict(n_groups=10, keep_groups=4, group_score="max"), dict(bias=bias)):
        check(mpe, l, 8, **kw)
        rows = [0, 1, 2, 3, 4, 7, 8, 9, 10, 11]
        check(mpe, l[rows], 8, score="sigmoid", **kw)
        check(mpe, l[rows], 8, score="sigmoid", renormalize=False, **kw)
    check(mpe, l[[2, 9, 10]], 8, score="sigmoid", bias=bias, n_groups=10, keep_groups=4)
    check(mpe, l[[2, 9, 10]], 8, score="sigmoid", bias=bias, n_groups=5, keep_groups=4, group_score="max")
    bias[8], bias[[20, 30]] = 0.0, INF
    check(mpe, l[9:], 8, score="sigmoid", bias=bias)
    check(mpe, l[9:], 8, bias=bias, n_groups=10, keep_groups=4)
    # far below zero a renormalised sigmoid still has its logits' ratios
    check(mpe, l[5:7].clamp(-500, -1), 8, score="sigmoid")


def test_strides_and_alignment(mpe):
    g = torch.Generator().manual_seed(7)
    full = torch.randn(40, 301, generator=g)
    for dtype in DT:
        f = full.to(DT[dtype]).cuda()
        for view in (f[:, :256], f[:, 1:257], f[:, 3:131], f[::3, :300], f[5:6, 2:66], f[:, 44:300]):
            check(mpe, view, 8)
    a = torch.randn(24, 320, generator=g).cuda()
    for view in (a[:, :256], a[:, 64:], a[:, 4:260], a[:, :192]):
        check(mpe, view, 8, score="sigmoid", bias=torch.randn(view.shape[1]).cuda() * 0.1)


def test_writes_only_its_rows(mpe):
    l = logits(7, 64)
    ids = torch.full((9, 6), -7, dtype=torch.int32, device="cuda")
    w = torch.full((9, 6), -7.0, device="cuda")
    mpe.select_experts(l, 6, ids=ids[1:8], w=w[1:8])
    assert (ids[[0, 8]] == -7).all() and (w[[0, 8]] == -7).all() and (ids[1:8] >= 0).all()


def test_on_another_stream_and_in_a_graph(mpe):
    l = logits(300, 256, seed=8)
    want = mpe.select_experts(l, 8, score=mpe.SCORE_SIGMOID)
    p_want = mpe.expert_importance(l)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        x = l * 1.0
        got = mpe.select_experts(x, 8, score=mpe.SCORE_SIGMOID)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    static = torch.zeros_like(l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ids, w = mpe.select_experts(static, 8, score=mpe.SCORE_SIGMOID)
        p = mpe.expert_importance(static)
    for _ in range(2):
        static.copy_(l)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1]) and torch.equal(p, p_want)


def test_every_16_bit_logit_in_order(mpe):
    """All bf16 and f16 values, signed zeros, infinities, subnormals and NaNs among them."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    order = torch.randperm(1 << 16, generator=torch.Generator().manual_seed(12))
    for dtype in (torch.bfloat16, torch.float16):
        l = bits[order].view(dtype).reshape(-1, 256).cuda()
        for score in ("softmax", "sigmoid"):
            l64 = l.double().cpu().numpy()
            for k, renorm in ((8, True), (32, False)):
                ids, w = mpe.select_experts(l, k, score=getattr(mpe, "SCORE_" + score.upper()), renormalize=renorm)
                assert np.array_equal(ids.cpu().numpy(), osel.select_experts(l64, k, score=score, renormalize=renorm)[0])
                broken = np.isnan(l64).any(axis=1) | (np.isposinf(l64).any(axis=1) if score == "softmax" else False)
                assert np.array_equal(torch.isnan(w).all(dim=1).cpu().numpy(), broken)
                assert np.array_equal(torch.isnan(w).any(dim=1).cpu().numpy(), broken)


def test_offsets_past_32_bits(mpe):
    """2.3e9 logits in one matrix, and rows 2^28 values apart."""
    T, E = 9_000_000, 256
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(13)
    rows = torch.tensor([0, 1, 8_388_607, 8_388_608, 8_388_609, T - 2, T - 1])
    l[rows.cuda()] = torch.randn(len(rows), E, generator=g).bfloat16().cuda()
    ids, w = mpe.select_experts(l, 1)
    rid, _ = osel.select_experts(l[rows.cuda()].double().cpu().numpy(), 1)
    assert np.array_equal(ids[rows.cuda()].cpu().numpy(), rid)
    assert int(ids.count_nonzero()) == int((rid != 0).sum())          # the rows of zeros choose expert 0
    # nearly every score is 1/256, summed over 9e6 tokens: the order of the sums decides nothing
    p = mpe.expert_importance(l).double().cpu().numpy()
    assert np.abs(p * E - 1).max() <= (256 + 17 + 80) * U + len(rows) * E / T
    flat = l.view(-1)[:8 * 2 ** 28]
    view = flat.view(8, 2 ** 28)[:, :E]
    view.copy_(torch.randn(8, E, generator=g).bfloat16())
    check(mpe, view, 8)
    check(mpe, view, 8, bias=torch.zeros(E).cuda())


@pytest.mark.parametrize("E", [1, 8, 33, 128, 200, 256, 500, 1024])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 100, 5000])
def test_importance(mpe, T, E):
    for dtype in ("f32", "bf16", "f16"):
        l = logits(T, E, dtype, seed=9)
        for score, name in ((mpe.SCORE_SOFTMAX, "softmax"), (mpe.SCORE_SIGMOID, "sigmoid")):
            p = mpe.expert_importance(l, score=score).double().cpu().numpy()
            l64 = l.double().cpu().numpy()
            ref = osel.expert_importance(l64, name)
            assert (np.abs(p - ref) <= importance_tol(l64, ref)).all()


@pytest.mark.parametrize("T,E", [(16, 1024), (17, 1024), (64, 256), (64, 257), (65, 8), (129, 1000), (256, 1024),
                                 (257, 1024), (512, 512), (512, 513), (513, 64)])
def test_importance_around_the_cluster(mpe, T, E):
    """Sizes on both sides of one CTA, a cluster of them and two launches; rows whole and not; two calls at once."""
    for dtype in ("f32", "f16"):
        for pad in (0, 3):
            l = torch.nn.functional.pad(logits(T, E, dtype, seed=14), (0, pad))[:, :E]
            l64 = l.double().cpu().numpy()
            ref = osel.expert_importance(l64, "softmax")
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            out = []
            for i in range(8):
                with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
                    out.append(mpe.expert_importance(l))
            torch.cuda.synchronize()
            assert all(torch.equal(out[0], p) for p in out)
            assert (np.abs(out[0].double().cpu().numpy() - ref) <= importance_tol(l64, ref)).all()


def test_importance_of_masked_and_broken_rows(mpe):
    l = logits(40, 64, seed=10)
    l[0] = -INF
    l[1, :60] = -INF
    for score, name in ((mpe.SCORE_SOFTMAX, "softmax"), (mpe.SCORE_SIGMOID, "sigmoid")):
        p = mpe.expert_importance(l, score=score).double().cpu().numpy()
        l64 = l.double().cpu().numpy()
        ref = osel.expert_importance(l64, name)
        assert (np.abs(p - ref) <= importance_tol(l64, ref)).all()
    l[2, 5] = float("nan")
    assert torch.isnan(mpe.expert_importance(l)).all()
    bad = torch.isnan(mpe.expert_importance(l, score=mpe.SCORE_SIGMOID))
    assert bad[5] and bad.sum() == 1
    l[2, 5] = INF
    assert torch.isnan(mpe.expert_importance(l)).all()
    assert torch.isfinite(mpe.expert_importance(l, score=mpe.SCORE_SIGMOID)).all()


def test_importance_repeats_to_the_bit_and_drives_the_allocator(mpe):
    l = logits(20000, 64, seed=11)
    p = mpe.expert_importance(l)
    assert torch.equal(p, mpe.expert_importance(l))
    assert abs(float(p.double().sum()) - 1.0) < 1e-5
    E, W = 64, 1 << 16
    bits = mpe.allocate_bits(p.cpu().numpy(), [W] * E, 5 * E * W)
    assert set(bits) <= {3, 4, 8} and int(bits.sum()) * W <= 5 * E * W
