"""The gated block, its gradients and the AdamW step as a training step of grouped
experts, then their weights in e4m3 as served: every result against 64-bit forms of
the values that went into it."""
import pytest
import torch

from block_util import STEP, adamw64, fp8_product64, gated64, quantise64, rand, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
M, D, F, E = 300, 256, 136, 4
OFFSETS = [0, 77, 77, 201, 290]


def ops():
    from sparse_mixture_experts_04_amd import ops
    return ops


class Trainer:
    """W_gate and W_up of E experts: fp32 parameters, bf16 copies that the block reads,
    bf16 gradients, states of `bits` bits; the gradient of h comes from outside."""

    def __init__(self, bits, act=BF):
        L = ops()
        self.bits = bits
        self.params = [rand((E, F, D), F32, s, D ** -0.5) for s in (1, 2)]
        self.weights = [p.to(act) for p in self.params] if act == BF else self.params
        self.grads = [torch.empty_like(w) for w in self.weights]
        zeros = lambda n, dt: [torch.zeros(n, dtype=dt, device="cuda") for _ in range(2)]
        shape, scales = (E, F, D), {}
        if bits == 8:
            n = (E * F * D + 255) // 256
            scales = dict(m_scales=zeros(n, F32), v_scales=zeros(n, F32))
        self.m, self.v = (zeros(shape, dt) for dt in
                          ((torch.int8, torch.uint8) if bits == 8 else (F32, F32)))
        self.scales = scales
        self.plan = L.adamw_plan(self.params, self.grads, self.m, self.v,
                                 copies=self.weights if act == BF else None, **scales)
        self.x, self.dh = rand((M, D), act, 3), rand((M, F), act, 4, 1e-2)
        self.h, self.dx = torch.zeros((M, F), dtype=act, device="cuda"), torch.zeros_like(self.x)
        self.pre = torch.empty((M, 2 * F), device="cuda")
        self.offsets = torch.tensor(OFFSETS, dtype=torch.int32, device="cuda")
        self.ws = L.gated_ff_workspace(M, D, F, E, act, "cuda", backward=True)
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.lr = torch.full((1,), 1e-2, device="cuda")
        self.factor = torch.full((1,), 0.25, device="cuda")

    def run(self):
        L = ops()
        self.step += 1
        L.gated_ff(self.x, *self.weights, self.h, offsets=self.offsets, pre=self.pre, ws=self.ws)
        L.gated_ff_backward(self.x, *self.weights, self.dh, self.dx, *self.grads,
                            offsets=self.offsets, pre=self.pre, ws=self.ws)
        L.adamw_step(self.plan, self.step, self.lr, grad_scale=self.factor, **HYPER)

    def state(self):
        all_ = dict(params=self.params, weights=self.weights, m=self.m, v=self.v, **self.scales)
        return {k: [t.clone() for t in l] for k, l in all_.items()}

    def check(self, old, step):
        want, covered = gated64(self.x, *old["weights"], OFFSETS, self.dh)
        rows = covered.cuda()
        for n, t in (("h", self.h[rows]), ("dx", self.dx[rows])):
            within(t, want[n][0][covered], want[n][1][covered], n)
        for n, t in zip(("dw_gate", "dw_up"), self.grads):
            within(t, *want[n], n)
        for i in range(2):
            kw = {k: old[n][i] for k, n in (("ms", "m_scales"), ("vs", "v_scales"))} if self.bits == 8 else {}
            r = adamw64(old["params"][i], self.grads[i], old["m"][i], old["v"][i], step,
                        float(self.lr), HYPER["beta1"], HYPER["beta2"], HYPER["eps"],
                        HYPER["weight_decay"], float(self.factor), **kw)
            within(self.params[i], r["p"], r["ep"], "p")
            if self.weights[i].dtype == BF:
                assert torch.equal(self.weights[i], self.params[i].to(BF))
            if self.bits == 8:
                assert torch.equal(self.m[i].cpu(), r["cm"]) and torch.equal(self.v[i].cpu(), r["cv"])
            else:
                within(self.m[i], r["m"], r["em"], "m")
                within(self.v[i], r["v"], r["ev"], "v")


@pytest.mark.parametrize("act", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bits", [32, 8])
def test_training_step(bits, act):
    t = Trainer(bits, act)
    for step in range(1, 4):
        old = t.state()
        t.run()
        t.check(old, step)
        t.x.copy_(rand(t.x.shape, act, 20 + step))


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step_captured(bits):
    """The step as a graph, replayed on new rows between eager work, against an eager
    trainer of the same inputs to the bit; the graph holds its own step count."""
    t, eager = Trainer(bits), Trainer(bits)
    start = t.state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run()
    t.step.zero_()
    for k, l in t.state().items():
        now = dict(params=t.params, weights=t.weights, m=t.m, v=t.v, **t.scales)[k]
        for a, b in zip(now, start[k]):
            a.copy_(b)
    for step in range(1, 5):
        for z in (t, eager):
            z.x.copy_(rand(t.x.shape, BF, 40 + step))
            z.lr.fill_(1e-2 / step)
        old = eager.state()
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        eager.check(old, step)
        a, b = t.state(), eager.state()
        for k in a:
            assert all(torch.equal(p, q) for p, q in zip(a[k], b[k])), (step, k)
        assert torch.equal(t.h, eager.h) and torch.equal(t.dx, eager.dx)


@pytest.mark.parametrize("rows", [3, 300])
def test_trained_weights_served_in_e4m3(rows):
    """Trained matrices quantised, then the two products of a batch with them."""
    L = ops()
    t = Trainer(32)
    for _ in range(2):
        t.run()
    x = rand((rows, D), BF, 99)
    codes, scales = L.quantize_fp8(x)
    want_codes, want_scales = quantise64(x)
    assert torch.equal(scales.cpu().double(), want_scales)
    g = codes.cpu().view(torch.uint8)
    assert ((g == want_codes) | ((g | want_codes) & 0x7f == 0)).all()
    edges = [0, 1, 1, 2, 3] if rows == 3 else OFFSETS
    off = torch.tensor(edges, dtype=torch.int32, device="cuda")
    for w in t.weights:
        wc, wsc = L.quantize_fp8_weights(w)
        y = torch.full((rows, F), 7.0, dtype=BF, device="cuda")
        L.gemm_fp8(codes, scales, wc, wsc, y, offsets=off)
        want, bound, covered = fp8_product64(codes, scales, wc, wsc, edges, BF)
        within(y[covered.cuda()], want[covered], bound[covered])
        assert (y.cpu()[~covered] == 7.0).all()
        # beside the product of the unquantised weights: each factor off by at most half
        # a step of e4m3, 2^-4 of it, and half its smallest step, 2^-10 of its scale
        X, W = x.cpu().double(), w.cpu().double()
        sx = want_scales.repeat_interleave(128, 1)[:, :D]
        sw = wsc.cpu().double().repeat_interleave(128, 1)[:, :F].repeat_interleave(128, 2)[:, :, :D]
        for e in range(E):
            lo, hi = edges[e], edges[e + 1]
            if lo == hi:
                continue
            ex = X[lo:hi].abs() / 16 + sx[lo:hi] * 2.0 ** -10
            ew = W[e].abs() / 16 + sw[e] * 2.0 ** -10
            off_by = ex @ W[e].abs().T + X[lo:hi].abs() @ ew.T + ex @ ew.T
            exact = X[lo:hi] @ W[e].T
            within(y[lo:hi], exact, off_by + bound[lo:hi], "against unquantised weights")
