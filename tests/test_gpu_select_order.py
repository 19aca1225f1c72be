"""The weights' normalising sum runs in the order of choice: a row whose experts stand in another order gives the
same weights to the bit, as do repeated calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mpe():
    import mixed_precision_expert_b200 as m
    m.lib()
    return m


@pytest.mark.parametrize("E", [32, 64, 100, 128, 256, 512, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_permuted_experts(mpe, E, score, with_bias):
    g = torch.Generator().manual_seed(E)
    # distinct logits in every row, far enough apart that no key ties
    l = torch.stack([torch.randperm(E, generator=g) for _ in range(500)]).float() * (8.0 / E) - 4.0
    l += torch.rand(l.shape, generator=g) * (4.0 / E)
    b = torch.randn(E, generator=g) * 0.1
    for k in (5, 8, 16, 32):
        kw = dict(score=getattr(mpe, "SCORE_" + score.upper()))
        ids, w = mpe.select_experts(l.cuda(), k, bias=b.cuda() if with_bias else None, **kw)
        for _ in range(3):
            p = torch.randperm(E, generator=g)
            ids2, w2 = mpe.select_experts(l[:, p].cuda(), k, bias=b[p].cuda() if with_bias else None, **kw)
            assert torch.equal(p.cuda()[ids2.long()].int(), ids)
            assert torch.equal(w2, w)
        for _ in range(3):
            again = mpe.select_experts(l.cuda(), k, bias=b.cuda() if with_bias else None, **kw)
            assert torch.equal(again[0], ids) and torch.equal(again[1], w)
