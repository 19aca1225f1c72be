"""mpe_select_experts with biases that are infinite or near the largest float32, against the float64 oracle: ids are
equal, weights as in test_gpu_select (the bias is not in them). Logits are columns of a wider buffer whose other
columns are NaN, so that an expert past the row shows."""
import numpy as np
import pytest
import torch

from oracle import select as osel

pytestmark = pytest.mark.gpu

INF = float("inf")
MAX = float(torch.finfo(torch.float32).max)
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mpe():
    import mixed_precision_expert_b200 as m
    m.lib()
    return m


def check(mpe, l, k, bias, score, **kw):
    T, E = l.shape
    wide = torch.full((T + 1, E + 5), float("nan"), dtype=l.dtype)
    wide[:T, :E] = l
    # behind the bias in its allocation, too: NaN
    b = torch.cat([bias, torch.full((64,), float("nan"))]).cuda()[:E]
    group_score = kw.pop("group_score", "top2")
    ids, w = mpe.select_experts(wide.cuda()[:T, :E], k, bias=b, score=getattr(mpe, "SCORE_" + score.upper()),
                                group_score=getattr(mpe, "GROUP_" + group_score.upper()), **kw)
    rid, rw = osel.select_experts(l.double().numpy(), k, bias=bias.double().numpy(), score=score,
                                  group_score=group_score, **kw)
    ids = ids.cpu().numpy()
    assert np.array_equal(ids, rid), (E, k, score, kw, np.argwhere(ids != rid)[:4])
    # spread of the logits below 20: (2 * 20 + 60) units
    assert (np.abs(w.double().cpu().numpy() - rw) <= np.abs(rw) * 100 * U + 2.0 ** -126).all()


def biases(E, g):
    """Mostly ordinary biases with one or several infinite or huge ones."""
    out = []
    for values in ((INF,), (-INF,), (INF, INF), (INF, -INF), (MAX,), (-MAX,), (MAX, MAX, -MAX), (2e38, -2e38, 2e38),
                   (-MAX, -INF), (INF, MAX, -MAX, -INF), (3e38, 3.2e38, 1e38)):
        for fill in ("randn", "zeros", "lowest"):
            b = torch.randn(E, generator=g) * 0.1 if fill == "randn" else torch.zeros(E)
            if fill == "lowest":
                b[:] = -MAX
            at = torch.randperm(E, generator=g)[:len(values)]
            b[at] = torch.tensor(values)[:len(at)]
            out.append(b)
    return out


@pytest.mark.parametrize("E", [1, 2, 5, 8, 20, 31, 32, 33, 64, 100, 256])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_infinite_and_huge_biases(mpe, E, score):
    g = torch.Generator().manual_seed(E)
    for n, b in enumerate(biases(E, g)):
        l = torch.randn(5, E, generator=g) * 1.5
        for k in sorted({1, min(E, 2), min(E, 4), min(E, 8)}):
            check(mpe, l, k, b, score)


@pytest.mark.parametrize("E,G,keep,k", [(14, 7, 3, 3), (14, 7, 2, 4), (30, 10, 7, 5), (32, 8, 3, 4), (32, 32, 8, 8), (31, 31, 9, 2),
                                        (20, 2, 1, 4), (32, 4, 2, 8), (6, 3, 2, 3), (64, 8, 3, 6), (256, 8, 4, 8)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_infinite_biases_in_groups(mpe, E, G, keep, k, score):
    """By the largest key: no sum that float32 could not hold."""
    g = torch.Generator().manual_seed(E * G)
    for b in biases(E, g):
        check(mpe, torch.randn(5, E, generator=g) * 1.5, k, b, score, n_groups=G, keep_groups=keep, group_score="max")


@pytest.mark.parametrize("E,G,keep,k", [(4, 2, 1, 2), (14, 7, 3, 3), (30, 10, 7, 5), (32, 8, 3, 4), (32, 32, 8, 8), (31, 31, 9, 2),
                                        (20, 2, 1, 4), (32, 4, 2, 8), (6, 3, 2, 3), (64, 8, 3, 6), (256, 8, 4, 8), (512, 16, 5, 8)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_sums_of_two_past_float32(mpe, E, G, keep, k, score):
    """Sums of a group's two largest keys that only float64 holds, beside true infinities."""
    g = torch.Generator().manual_seed(E * G + 1)
    more = []
    for values in ((2e38, 2e38, 3e38, 3e38), (-2e38, -3e38, -3.4e38), (-MAX, -INF), (MAX, 3e38, 2e38, -INF)):
        more.append(torch.tensor(values)[torch.randint(0, len(values), (E,), generator=g)])
    # one usable expert in some groups, all barred by the lowest float in others
    b = torch.full((E,), -MAX)
    b[::3] = -INF
    more.append(b)
    # whole groups barred, which is common: the rest by their scores
    b = torch.randn(E, generator=g) * 0.1
    b[E // G * ((G + 1) // 2):] = -INF
    more.append(b)
    for b in biases(E, g) + more:
        with np.errstate(invalid="ignore"):  # inf - inf in a group's sum: NaN, which ranks lowest
            check(mpe, torch.randn(5, E, generator=g) * 1.5, k, b, score, n_groups=G, keep_groups=keep)


def test_the_larger_of_two_sums_past_float32(mpe):
    b = torch.tensor([2e38, 2e38, 3e38, 3e38])
    check(mpe, torch.zeros(3, 4), 2, b, "sigmoid", n_groups=2, keep_groups=1)
    check(mpe, torch.zeros(3, 4), 2, -b.flip(0), "sigmoid", n_groups=2, keep_groups=1)
