"""The few-token layer's gates at logits of any finite size, and the precision of
its sums."""
import pytest
import torch

import int8_util as R
import test_few_gpu as few_tests
from sparse_mixture_experts_04_amd.configs import MoEConfig

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("sign", ["both", "negative"])
@pytest.mark.parametrize("form", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("xs,ws", [(1e2, 1e1), (1e6, 1e25), (1e10, 1e36), (1e18, 1e37)])
def test_logsumexp_gates_of_huge_logits(xs, ws, form, sign):
    """Logits up to 1e57 (finite x and w_router): contributors far below the largest
    have gate 0, and every gate is finite.  Negative: all affinities are 0, the bias
    alone picks, and the gates come from logits that lie as far apart."""
    print(f"huge logits x {xs} w {ws} {form} {sign}", flush=True)
    cfg = MoEConfig("few_huge", T=16, d=256, F=128, act="f32" if form == "f32" else "bf16", E=64,
                    S=2, bias_range=0.05)
    inp = few_tests.layer(cfg)
    inp["x"] *= xs
    inp["w_router"] *= ws
    if sign == "negative":
        inp["x"].abs_()
        inp["w_router"].abs_().neg_()
    for n in ("w_gate", "w_up", "ws_gate", "ws_up"):    # the experts' products stay near 1
        inp[n] /= xs
    desc = few_tests.L.make_desc(cfg.T, cfg.d, cfg.F, inp["x"].dtype, E=cfg.E, S=cfg.S,
                                 gate_norm="logsumexp", gate_scale=2.0)
    int8 = form == "int8"
    w, q = few_tests.L.int8_weights(inp) if int8 else (few_tests.L.weights_from(inp), inp)
    y, idx, g = few_tests.few(desc, inp, w)
    assert torch.isfinite(g).all()
    _, g64 = R.route64(inp["x"], inp["w_router"], inp["bias"], cfg.S, "logsumexp", 2.0)
    # below fp32's normal range a gate may be off by its smallest step
    assert ((g.double() - g64).abs() <= (R.EPS32 + 1e-12) * g64.abs() + 2.0 ** -149).all()
    few_tests.check(cfg, desc, inp, q, int8, y, idx, g64, gate_norm="logsumexp", gate_scale=2.0)


def layer_on_cpu(inp, S, h_of=lambda h: h):
    """The layer in float64 on the CPU, with h_of applied to h before the down
    product; only the experts that are picked are copied."""
    x = inp["x"].cpu()
    idx, g = (v.cpu() for v in R.route64(inp["x"], inp["w_router"], inp["bias"], S))

    def expert(kind, e, rows):
        wg, wu, wd = (inp[f"{kind}_{p}"][e].cpu().double() for p in ("gate", "up", "down"))
        v = x[rows].double()
        y = h_of(R.silu64(v @ wg.t()) * (v @ wu.t())) @ wd.t()
        return y, torch.zeros_like(y)
    return R.layer64(x, idx, g, expert, S)[0]


# T, d, F, E, S: one pass over K in either stage, then several in the down stage, in both
PRECISION = [(1, 512, 128, 256, 2), (2, 768, 256, 128, 1), (8, 2048, 768, 256, 2),
             (16, 512, 384, 64, 2), (3, 256, 16384, 64, 1), (16, 256, 8192, 64, 2),
             (16, 4096, 3200, 64, 1)]


def sum_error(d, F):
    """Expected error of y relative to its size from fp32 sums of random terms: a
    lane of the wave adds every 64th term or group of terms one after another, half
    a step for each square root of their number, and 6 exchanges add the lanes (up
    to 3 half steps in all); the gate and up sums reach h through silu and the
    product by a factor of at most 3."""
    return (3 * (d / 64) ** 0.5 + (F / 64) ** 0.5 + 3) * R.EPS32


@pytest.mark.parametrize("T,d,F,E,S", PRECISION)
def test_bf16_layer_keeps_h_to_17_bits(T, d, F, E, S):
    """h enters the down product to 2^-17.  A y whose error is e steps of bf16
    (small e) rounds to another value than the exact y with probability e.  With
    errors of r times y's size, normal ys and steps of at least 2^-8 of y that
    makes 0.8 a (1.1 + ln 1/a) of the values, a = 0.8 * 2^8 r.  h rounded once to
    bf16 would change two values in five."""
    print(f"few precision T={T} d={d} F={F} S={S}", flush=True)
    inp = few_tests.gpu_layer(T, d, F, E, S, "bf16", 3 * T + d + F)
    desc = few_tests.L.make_desc(T, d, F, torch.bfloat16, E=E, S=S)
    y = few_tests.few(desc, inp, few_tests.L.weights_from(inp))[0].cpu()
    exact = layer_on_cpu(inp, S)
    a = 0.8 * 2 ** 8 * (2.0 ** -17 + sum_error(d, F))
    share = 0.8 * a * (1.1 + torch.log(torch.tensor(1 / a)).item())
    limit = share + 5 * (share / y.numel()) ** 0.5
    other = (y != exact.to(torch.bfloat16)).double().mean().item()
    once = layer_on_cpu(inp, S, lambda h: h.to(torch.bfloat16).double()).to(torch.bfloat16)
    planted = (once != exact.to(torch.bfloat16)).double().mean().item()
    print(f"   other roundings {other:.4f}, limit {limit:.4f}, h rounded once {planted:.3f}",
          flush=True)
    assert other <= limit
    assert planted > 4 * limit          # the limit tells the two apart


@pytest.mark.parametrize("T,d,F,E,S", PRECISION)
def test_f32_layer_errors_are_those_of_random_sums(T, d, F, E, S):
    """Twice the expected error (see sum_error), and the rounding of y."""
    print(f"few precision f32 T={T} d={d} F={F} S={S}", flush=True)
    inp = few_tests.gpu_layer(T, d, F, E, S, "f32", 3 * T + d + F)
    desc = few_tests.L.make_desc(T, d, F, torch.float32, E=E, S=S)
    y = few_tests.few(desc, inp, few_tests.L.weights_from(inp))[0].cpu().double()
    exact = layer_on_cpu(inp, S)
    rel = ((y - exact).norm(dim=1) / exact.norm(dim=1)).max().item()
    limit = 2 * sum_error(d, F) + R.EPS32
    print(f"   rel L2 {rel:.2e}, limit {limit:.2e}", flush=True)
    assert rel <= limit
