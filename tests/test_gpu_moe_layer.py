"""The operators around the routed experts run together, as a layer uses them:
router projection -> choice of experts -> routed experts from pages -> shared
expert added to their output; and importances -> widths."""
import numpy as np
import pytest
import torch

import synth
from oracle import linear as oln
from oracle import select as osel
from tests._helpers import check_ffn, oracle_moe, OracleExpert, workload_masters_cpu, workload_masters_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    import mixed_precision_expert_b200 as mpe
    wl = synth.WORKLOADS[1]
    g = torch.Generator().manual_seed(77)
    E, H, F = wl.E, wl.H, wl.F
    router = (torch.randn(E, H, generator=g) / H ** 0.5 * 2).bfloat16()
    shared_in = (torch.randn(2 * F, H, generator=g) / H ** 0.5).bfloat16()
    shared_out = (torch.randn(H, F, generator=g) / F ** 0.5).bfloat16()
    masters = workload_masters_gpu(wl)
    # importances over a calibration batch decide the widths
    calib = torch.randn(4000, H, generator=g).bfloat16().cuda()
    p = mpe.expert_importance(mpe.linear(calib, router.cuda(), out_dtype=torch.float32)).cpu().numpy()
    bits = mpe.allocate_bits(p, [wl.W_e] * E, wl.budget_bits)
    ctx = mpe.Context(E, H, F)
    ctx.quantize_experts(masters, bits)
    mats = {e: OracleExpert(workload_masters_cpu(wl, e), H, F, int(bits[e])).mats() for e in range(E)}
    yield mpe, wl, ctx, router, shared_in, shared_out, mats
    ctx.close()


def forward(mpe, ctx, x, router, shared_in, shared_out, k):
    logits = mpe.linear(x, router, out_dtype=torch.float32)
    ids, w = mpe.select_experts(logits, k)
    y = ctx.moe_ffn(x, ids, w)
    h = mpe.linear(x, shared_in, act=mpe.ACT_SILU, gated=True)
    mpe.linear(h, shared_out, residual=y, out=y)
    return logits, ids, w, y


@pytest.mark.parametrize("T", [1, 3, 64, 300])
def test_layer(layer, T):
    mpe, wl, ctx, router, shared_in, shared_out, mats = layer
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, wl.H, generator=g).bfloat16()
    dev = [t.cuda() for t in (router, shared_in, shared_out)]
    logits, ids, w, y = forward(mpe, ctx, x.cuda(), *dev, wl.k)
    torch.cuda.synchronize()
    x64 = x.double().numpy()
    ref_logits = oln.linear(x64, router.double().numpy())
    # H float32 additions in any order, each off by 2^-23 of what they add up to at most
    room = wl.H * 2.0 ** -23 * (np.abs(x64) @ np.abs(router.double().numpy()).T)
    assert (np.abs(logits.double().cpu().numpy() - ref_logits) <= room).all()
    # the choice is the oracle's for the logits that the projection gave
    rid, rw = osel.select_experts(logits.double().cpu().numpy(), wl.k)
    assert np.array_equal(ids.cpu().numpy(), rid)
    routed = oracle_moe(x, rid, rw, lambda e: mats[e], wl.E)
    h = oln.linear(x64, shared_in.double().numpy(), act="silu", gated=True)
    check_ffn(y.double().cpu().numpy(), oln.linear(h, shared_out.double().numpy(), residual=routed))
    assert ctx.status() == 0 and mpe.global_status() == 0


def test_layer_in_a_graph(layer):
    mpe, wl, ctx, router, shared_in, shared_out, _ = layer
    dev = [t.cuda() for t in (router, shared_in, shared_out)]
    xs = [torch.randn(32, wl.H, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(3)]
    want = [forward(mpe, ctx, x, *dev, wl.k)[3].clone() for x in xs]
    static = torch.zeros_like(xs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(mpe, ctx, static, *dev, wl.k)[3]
    for x, y in zip(xs, want):
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)


def test_repage_from_importances(layer):
    mpe, wl, ctx, router, *_ = layer
    x = torch.randn(500, wl.H, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    p = mpe.expert_importance(mpe.linear(x, router.cuda(), out_dtype=torch.float32)).cpu().numpy()
    before = ctx.bits().copy()
    ctx.repage(4 * wl.E * wl.W_e, p)
    after = ctx.bits()
    assert int(after.astype(np.int64).sum()) <= 4 * wl.E
    ctx.repage(wl.budget_bits, p)
    assert ctx.bits().shape == before.shape and ctx.status() == 0


def test_binding_checks():
    import mixed_precision_expert_b200 as mpe
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
    l = z(4, 64)
    bad = [lambda: mpe.select_experts(l.double(), 4), lambda: mpe.select_experts(z(64, 4).t(), 4),
           lambda: mpe.select_experts(l[0], 4), lambda: mpe.select_experts(l, 4, bias=z(63)),
           lambda: mpe.select_experts(l, 4, bias=z(64).half()), lambda: mpe.select_experts(l, 4, bias=z(128)[::2]),
           lambda: mpe.select_experts(l, 4, bias=torch.zeros(64)), lambda: mpe.select_experts(l, 4, ids=z(4, 4)),
           lambda: mpe.select_experts(l, 4, w=z(4, 5)), lambda: mpe.select_experts(l, 4, w=z(4, 8)[:, ::2]),
           lambda: mpe.select_experts(l, 4, w=z(4, 4).half()), lambda: mpe.expert_importance(l.int()),
           lambda: mpe.expert_importance(l, out=z(64).double()), lambda: mpe.expert_importance(l, out=z(63))]
    bf = torch.bfloat16
    x, w = z(4, 64, dt=bf), z(128, 64, dt=bf)
    for kw in (dict(x=x.half()), dict(x=x[:, :32]), dict(x=z(64, 4, dt=bf).t()), dict(weight=w[:, :32]),
               dict(weight=w.cpu()), dict(weight=w[:127], gated=True), dict(bias=z(64)), dict(bias=z(128).half()),
               dict(out=z(4, 127)), dict(out=z(4, 128), out_dtype=bf), dict(residual=z(4, 128), out_dtype=bf),
               dict(residual=z(5, 128)), dict(out=z(4, 128).double()), dict(residual=z(4, 128, dt=bf)[0])):
        bad.append(lambda kw=kw: mpe.linear(**{"x": x, "weight": w, **kw}))
    for call in bad:
        with pytest.raises(ValueError):
            call()
    # what the library itself refuses
    wide = z(6, 72, dt=bf)
    for call in (lambda: mpe.select_experts(l, 65), lambda: mpe.select_experts(l, 4, n_groups=3),
                 lambda: mpe.linear(x.float(), w.float()), lambda: mpe.linear(wide[:4, 1:65], w),
                 lambda: mpe.linear(z(6, 68, dt=bf)[:4, :64], w), lambda: mpe.linear(x, w, out=w[:8].view(4, 128)),
                 lambda: mpe.linear(x, w, act=9)):
        with pytest.raises(mpe.MpeError) as e:
            call()
        assert e.value.code == -1
    assert mpe.select_experts(l[:0], 4)[0].shape == (0, 4)
    assert mpe.linear(x[:0], w).shape == (0, 128)
