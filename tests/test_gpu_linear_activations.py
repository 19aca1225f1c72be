"""mpe_linear's activations over their whole range, tails too, relative to the value itself, against float64.

v = x0 w + x1 w is exact in float32 (16 bits of x0 + x1, w a power of two), so all that is off is the activation, in
units of u = 2^-24 of the value:

  gelu      float32 results: erfc is off by 4 ulp (8 u); its argument, by a constant's and a product's rounding (1.3 u),
            moves it by at most v^2 + 1 times that; two products: 1.3 v^2 + 12.
            16-bit: the fit 15 u, rcp and ex2 (1 and 2 ulp) 6 u, nine roundings of the polynomial and products, the
            exponent's argument, v^2 / 2 with two roundings and a constant's (2.3 u): 1.2 v^2 + 31.
  silu      float32: e^-|v| (2 ulp, 4 u) moves e / (1 + e) by 1 / (1 + e) and 1 / (1 + e) by e / (1 + e) times that, 4 u
            at most; a sum 1 u, a quotient (2 ulp) 4 u, a product 1 u: 10.
            16-bit: the exponential 2 + 1.2 |v| ulp, rcp 1 ulp, a sum, a product: 2.4 |v| + 9.
  gelu_tanh as silu at z = 2 sqrt(2 / pi) (v + 0.044715 v^3), whose six roundings move the result by |z| each at most.

A 16-bit result is rounded once: half a step of its binade (of the smallest normal's below that). Values below
float32's smallest normal may be flushed to zero on the way (2^-126 |v| and the last product)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mpe():
    import mixed_precision_expert_b200 as m
    m.lib()
    return m


def values():
    v = torch.cat([torch.linspace(-14, 14, 3001), torch.logspace(-6, 1, 500), -torch.logspace(-6, 1, 500),
                   torch.tensor([0.0, -0.0, 20.0, -20.0, 60.0, -60.0, -88.0, 88.0])])
    hi = v.bfloat16()
    return hi, (v - hi.float()).bfloat16()


def form(v, act):
    """(value, z: the sigmoid's argument) in float64."""
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0)), v
    z = v if act == "silu" else math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3)
    return v / (1.0 + torch.exp(-z)), z


def units(v, z, act, out):
    if act == "gelu":
        return 1.3 * v * v + 12 if out == "f32" else 1.2 * v * v + 31
    fast = 10 if out == "f32" else 2.4 * z.abs() + 9
    return fast + (6 * z.abs() if act == "gelu_tanh" else 0)


def run(mpe, act, out, N, K, gated):
    hi, lo = values()
    x = torch.zeros(len(hi), K, dtype=DT["bf16"])
    x[:, 0], x[:, 1] = hi, lo
    if out == "f16":
        x = torch.where(x.abs() < 2.0 ** -14, 0.0, x.float()).half()  # normal values; 8 bits each
    w = torch.zeros(2 * N if gated else N, K, dtype=x.dtype)
    w[:N, :2] = torch.tensor([1.0, -1.0, 0.5, -0.5])[torch.arange(N) % 4][:, None]
    if gated:
        w[N:, 2] = 1.0
        x[:, 2] = 1.0  # up projection: 1
    got = mpe.linear(x.cuda(), w.cuda(), act=getattr(mpe, "ACT_" + act.upper()), gated=gated, out_dtype=DT[out])
    v = x.double() @ w[:N].double().t()
    assert torch.equal(v, v.float().double())
    ref, z = form(v, act)
    tol = ref.abs() * units(v, z, act, out) * U + (v.abs() + 1) * 2.0 ** -126
    if out != "f32":
        binade = torch.clamp(ref.abs() + tol, min=torch.finfo(DT[out]).tiny).log2().floor().exp2()
        tol = tol + binade * torch.finfo(DT[out]).eps / 2
    off = (got.double().cpu() - ref).abs()
    bad = off > tol
    assert not bad.any(), (int(bad.sum()), v[bad][:5], ref[bad][:5], got.cpu()[bad][:5])


@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K,gated", [(4, 16, False), (5, 16, False), (512, 64, False), (1028, 64, True)])
def test_relative_to_the_value(mpe, act, out, N, K, gated):
    run(mpe, act, out, N, K, gated)
