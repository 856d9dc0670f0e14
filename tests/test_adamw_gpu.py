"""The AdamW step against its formula in 64 bits."""
import pytest
import torch

from block_util import STEP, adamw64, rand, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def ops():
    from sparse_mixture_experts_04_amd import ops
    return ops


def ref(p, g, m, v, step, factor=1.0, ms=None, vs=None, **kw):
    h = {**HYPER, **kw}
    return adamw64(p, g, m, v, step, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"],
                   factor, ms, vs)


def tensors(sizes, pt, gt, bits, seed=0, skew=0, values=False):
    t = {"params": [rand((n,), pt, seed + 10 * i, 0.05, skew=skew) for i, n in enumerate(sizes)],
         "grads": [rand((n,), gt, seed + 10 * i + 1, 1e-3, skew=skew) for i, n in enumerate(sizes)]}
    if bits == 32:
        t["exp_avg"] = [rand((n,), F32, seed + 10 * i + 2, 1e-3, skew=skew) for i, n in enumerate(sizes)]
        t["exp_avg_sq"] = [rand((n,), F32, seed + 10 * i + 3, 1e-3, skew=skew).square_()
                           for i, n in enumerate(sizes)]
        return t
    g = torch.Generator().manual_seed(seed)
    code = lambda n, lo, hi, dt: torch.randint(lo, hi, (n + skew,), generator=g).to(dt).cuda()[skew:]
    t["exp_avg"] = [code(n, -127, 128, torch.int8) for n in sizes]
    t["exp_avg_sq"] = [code(n, 1, 256, torch.uint8) for n in sizes]
    sc = lambda n, s: ((torch.rand((n + 255) // 256, generator=g) + 0.5) * s).cuda()
    t["m_scales"] = [sc(n, 1e-3) for n in sizes]
    t["v_scales"] = [sc(n, 1e-6) for n in sizes]
    if values:
        t["m_values"] = [torch.full((n,), 9.0, device="cuda") for n in sizes]
        t["v_values"] = [torch.full((n,), 9.0, device="cuda") for n in sizes]
    return t


def clone(t):
    return {k: [x.clone() for x in v] for k, v in t.items()}


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 40961]


def check(t, old, step, factor=1.0, copies=None, **kw):
    for i in range(len(t["params"])):
        o = {k: v[i] for k, v in old.items()}
        r = ref(o["params"], o["grads"], o["exp_avg"], o["exp_avg_sq"], step, factor,
                o.get("m_scales"), o.get("v_scales"), **kw)
        pt = t["params"][i].dtype
        extra = STEP[BF] * (r["p"].abs() + r["ep"]) if pt == BF else 0.0
        within(t["params"][i], r["p"], r["ep"] + extra, f"p[{i}]")
        if copies is not None:
            assert torch.equal(copies[i], t["params"][i].to(BF))
        if "cm" in r:
            assert torch.equal(t["exp_avg"][i].cpu(), r["cm"]), f"m codes of {i}"
            assert torch.equal(t["exp_avg_sq"][i].cpu(), r["cv"]), f"v codes of {i}"
            # the largest value, rounded to fp32 (its 64-bit sum may round either way)
            within(t["m_scales"][i], r["s"].double(), r["s"].double() * 2.0 ** -23 + 1e-44)
            within(t["v_scales"][i], r["z"].double(), r["z"].double() * 2.0 ** -23 + 1e-44)
        else:
            within(t["exp_avg"][i], r["m"], r["em"], f"m[{i}]")
            within(t["exp_avg_sq"][i], r["v"], r["ev"], f"v[{i}]")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", [BF, F32], ids=["gbf16", "gf32"])
@pytest.mark.parametrize("pt", [BF, F32], ids=["pbf16", "pf32"])
def test_step(pt, gt, bits):
    L = ops()
    t = tensors(SIZES, pt, gt, bits, values=bits == 8)
    old = clone(t)
    copies = [torch.zeros(n, dtype=BF, device="cuda") for n in SIZES] if pt == F32 else None
    plan = L.adamw_plan(**t, copies=copies)
    L.adamw_step(plan, 17, **HYPER)
    check(t, old, 17, copies=copies)
    if bits == 8:
        L.adamw_state_values(plan)
        for i, n in enumerate(SIZES):
            s, z = (x[i].double().repeat_interleave(256)[:n] for x in (t["m_scales"], t["v_scales"]))
            c, q = t["exp_avg"][i].double(), t["exp_avg_sq"][i].double()
            # the value, rounded once (its 64-bit product may round either way)
            for got, v in ((t["m_values"][i], s * c * c.abs() / 127.0 ** 2),
                           (t["v_values"][i], z * q ** 4 / 255.0 ** 4)):
                within(got, v.cpu(), 2.0 ** -23 * v.abs().cpu())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("skew", [1, 3, 4])
def test_unaligned(skew, bits):
    L = ops()
    for pt, gt in ((F32, F32), (BF, BF), (F32, BF)):
        t = tensors([300, 2048, 4500], pt, gt, bits, skew=skew)
        old = clone(t)
        L.adamw_step(L.adamw_plan(**t), 3, **HYPER)
        check(t, old, 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More tensors than one table launch takes, empty ones among them."""
    L = ops()
    g = torch.Generator().manual_seed(1)
    sizes = torch.randint(0, 3000, (150,), generator=g).tolist()
    sizes[:3], sizes[70], sizes[-2:] = [0, 0, 5], 0, [0, 0]
    t = tensors(sizes, F32, F32, bits)
    old = clone(t)
    L.adamw_step(L.adamw_plan(**t), 2, **HYPER)
    check(t, old, 2)


def test_only_empty_tensors():
    L = ops()
    L.adamw_step(L.adamw_plan(**tensors([0, 0], F32, F32, 32)), 1, **HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero_states(bits):
    """Steps 1 to 5 from states of zeros, each against the formula on the states before."""
    L = ops()
    t = tensors([1000, 513], F32, F32, bits)
    for k in t:
        if k not in ("params", "grads"):
            for x in t[k]:
                x.zero_()
    plan = L.adamw_plan(**t)
    for step in range(1, 6):
        for i, g in enumerate(t["grads"]):
            g.copy_(rand(g.shape, F32, 100 * step + i, 1e-3))
        old = clone(t)
        L.adamw_step(plan, step, **HYPER)
        check(t, old, step)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients(bits):
    """Zero gradients on zero states: p only decays, nothing becomes NaN."""
    L = ops()
    t = tensors([700], F32, F32, bits)
    for k in t:
        if k != "params":
            t[k][0].zero_()
    old = clone(t)
    L.adamw_step(L.adamw_plan(**t), 1, **HYPER)
    check(t, old, 1)
    assert all(torch.isfinite(x.float()).all() for v in t.values() for x in v)


def test_small_v_stays_positive():
    """A v far below its block's largest keeps the smallest code, not 0."""
    L = ops()
    t = tensors([256], F32, F32, 8)
    for k in ("exp_avg", "exp_avg_sq", "m_scales", "v_scales"):
        t[k][0].zero_()
    t["grads"][0].fill_(1e-9)
    t["grads"][0][3] = 1.0
    old = clone(t)
    L.adamw_step(L.adamw_plan(**t), 1, **HYPER)
    check(t, old, 1)
    assert (t["exp_avg_sq"][0][:3] == 1).all()


def test_codes_at_borders():
    """Gradients that put |m'| and v' on and beside every border between two codes."""
    L = ops()
    k = torch.arange(127, dtype=torch.float64)
    m = ((k + 0.5) / 127) ** 2
    around = torch.cat([m * (1 + e) for e in (0, 1e-7, -1e-7, 3e-5, -3e-5)])
    n = (around.numel() + 254) // 255
    g = torch.zeros(n * 256)
    g.view(n, 256)[:, 0] = 1.0
    flat = torch.zeros(n * 255)
    flat[:around.numel()] = around.float()
    g.view(n, 256)[:, 1:] = flat.view(n, 255)
    for power in (1.0, 0.5):   # v' = g^2: its borders at the roots
        grad = (g ** power).cuda()
        t = {"params": [torch.zeros(n * 256, device="cuda")], "grads": [grad],
             "exp_avg": [torch.zeros(n * 256, dtype=torch.int8, device="cuda")],
             "exp_avg_sq": [torch.zeros(n * 256, dtype=torch.uint8, device="cuda")],
             "m_scales": [torch.zeros(n, device="cuda")], "v_scales": [torch.zeros(n, device="cuda")]}
        old = clone(t)
        L.adamw_step(L.adamw_plan(**t), 1, **HYPER)
        check(t, old, 1)


def test_not_finite_gradient():
    """32 bits: its own values only.  8 bits: its block of 256."""
    L = ops()
    for bad in (float("nan"), float("inf")):
        t = tensors([1000], F32, F32, 32)
        old = clone(t)
        t["grads"][0][300] = bad
        L.adamw_step(L.adamw_plan(**t), 5, **HYPER)
        ok = torch.isfinite(t["params"][0])
        assert not ok[300] and ok.sum() == 999
        t = tensors([1000], F32, F32, 8)
        old = clone(t)
        t["grads"][0][300] = bad
        L.adamw_step(L.adamw_plan(**t), 5, **HYPER)
        assert torch.isnan(t["m_scales"][0]).tolist() == [False, True, False, False]
        assert torch.isnan(t["v_scales"][0]).tolist() == [False, True, False, False]
        assert not t["exp_avg"][0][256:512].any() and not t["exp_avg_sq"][0][256:512].any()
        ok = torch.isfinite(t["params"][0])
        assert not ok[300] and ok.sum() == 999


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale(bits):
    L = ops()
    for f in (0.37, 0.0):
        t = tensors([3000], F32, BF, bits)
        old = clone(t)
        factor = torch.tensor([f], device="cuda")
        L.adamw_step(L.adamw_plan(**t), 9, **HYPER, grad_scale=factor)
        check(t, old, 9, factor=float(factor))
    for f in (float("nan"), float("inf"), -float("inf")):
        t = tensors([3000], F32, BF, bits)
        old = clone(t)
        L.adamw_step(L.adamw_plan(**t), 9, **HYPER, grad_scale=torch.tensor(f, device="cuda"))
        for k in t:
            assert torch.equal(t[k][0], old[k][0]), k


def test_other_hyper_parameters():
    L = ops()
    for kw in (dict(beta1=0.0), dict(beta2=0.999), dict(eps=0.1), dict(weight_decay=0.0),
               dict(lr=0.0), dict(lr=-1e-3), dict(beta1=0.95, beta2=0.0, eps=1e-3)):
        t = tensors([3000], F32, F32, 32)
        old = clone(t)
        L.adamw_step(L.adamw_plan(**t), 40, **{**HYPER, **kw})
        check(t, old, 40, **kw)


def test_captured_with_step_and_rate_on_the_gpu():
    """A replayed graph follows the step counter and the rate; each replay against the
    formula on the states before it."""
    L = ops()
    for bits in (32, 8):
        t = tensors([5000, 77], F32, BF, bits)
        plan = L.adamw_plan(**t)
        step = torch.zeros(1, dtype=torch.int64, device="cuda")
        lr = torch.zeros(1, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step += 1
            L.adamw_step(plan, step, **{**HYPER, "lr": lr})
        step.zero_()
        for i in range(1, 4):
            lr.fill_(1e-3 / i)
            for j, g in enumerate(t["grads"]):
                g.copy_(rand(g.shape, BF, 50 * i + j, 1e-3))
            old = clone(t)
            graph.replay()
            torch.cuda.synchronize()
            assert int(step) == i
            check(t, old, i, lr=float(lr))


def test_shapes_and_a_second_plan():
    """Matrices of any shape; the same tensors under two plans."""
    L = ops()
    t = {"params": [rand((3, 40, 65), F32, 1), rand((9,), F32, 2)],
         "grads": [rand((3, 40, 65), F32, 3), rand((9,), F32, 4)],
         "exp_avg": [torch.zeros((3, 40, 65), device="cuda"), torch.zeros(9, device="cuda")],
         "exp_avg_sq": [torch.zeros((3, 40, 65), device="cuda"), torch.zeros(9, device="cuda")]}
    old = clone(t)
    L.adamw_step(L.adamw_plan(**t), 1, **HYPER)
    check(t, old, 1)
    old = clone(t)
    L.adamw_step(L.adamw_plan(**t), 2, **HYPER)
    check(t, old, 2)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size,eps", [(1e-17, 0.0), (1e-20, 1e-8), (1e-30, 1e-8), (1e18, 1e-8)])
def test_sizes_of_gradients(size, eps, bits):
    """Scales far from 1: roots beyond the reach of the short forms, values below the
    smallest normal fp32, squares near its largest."""
    L = ops()
    t = tensors([3000, 77], F32, F32, bits)
    for k in ("exp_avg", "exp_avg_sq", "m_scales", "v_scales"):
        for x in t.get(k, []):
            x.zero_()
    plan = L.adamw_plan(**t)
    for step in (1, 2):
        for i, g in enumerate(t["grads"]):
            z = rand(g.shape, F32, 7 * step + i)      # half of `size` to some 4 of it
            g.copy_((torch.sign(z) * 0.5 + z) * size)
        old = clone(t)
        L.adamw_step(plan, step, **{**HYPER, "eps": eps})
        check(t, old, step, eps=eps)


def test_values_without_a_place_for_them():
    """The table's tensors without m_values are passed over, their neighbours not."""
    import ctypes
    L = ops()
    from sparse_mixture_experts_04_amd import _lib
    t = tensors([3000], F32, F32, 8)
    plan = L.adamw_plan(**t)
    before = clone(t)
    with pytest.raises(ValueError):
        L.adamw_state_values(plan)
    status = _lib.lib.moe_adamw_state_values(ctypes.byref(plan.desc), plan.chunks,
                                             plan.table.data_ptr(), None)
    torch.cuda.synchronize()
    assert status == 0
    for k in t:
        assert torch.equal(t[k][0], before[k][0]), k


def test_step_on_another_stream():
    """A plan made on one stream, its steps on another at once."""
    L = ops()
    t = tensors([70000, 5], F32, BF, 8)
    old = clone(t)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = L.adamw_plan(**t)
    with torch.cuda.stream(s):
        L.adamw_step(plan, 4, **HYPER)
    s.synchronize()
    check(t, old, 4)


def test_same_bits_again():
    L = ops()
    for bits in (32, 8):
        t = tensors([100000], BF, F32, bits)
        u = clone(t)
        for x in (t, u):
            L.adamw_step(L.adamw_plan(**x), 6, **HYPER)
        for k in t:
            assert torch.equal(t[k][0], u[k][0]), (bits, k)


def test_refusals_of_the_binding():
    L = ops()
    t = tensors([300, 20], F32, F32, 32)
    e = tensors([300, 20], F32, F32, 8)
    bad = [{**t, "params": [t["params"][0]] * 2}, {**t, "grads": t["grads"][:1]},
           {**t, "grads": [t["grads"][0], t["grads"][1].to(BF)]},
           {**t, "params": [t["params"][0], t["params"][1].half()]},
           {**t, "exp_avg": [t["exp_avg"][0], t["exp_avg"][1][:10]]},
           {**t, "exp_avg_sq": [x.double() for x in t["exp_avg_sq"]]},
           {**t, "m_scales": e["m_scales"], "v_scales": e["v_scales"]},
           {**t, "copies": [x.clone() for x in t["params"]]},
           {**e, "m_scales": None}, {**e, "v_scales": [x[:1] for x in e["v_scales"]]},
           {**e, "exp_avg_sq": e["exp_avg"]}, {**e, "m_values": [x.clone() for x in e["params"]]},
           {**t, "params": [x.cpu() for x in t["params"]]},
           {**t, "params": [t["params"][0], t["params"][0][5:25]]}]
    for kw in bad:
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            L.adamw_plan(**kw)
    bf = tensors([300], BF, F32, 32)
    with pytest.raises(RuntimeError):                               # copies of bf16 parameters
        L.adamw_plan(**bf, copies=[x.clone() for x in bf["params"]])
    plan, old = L.adamw_plan(**t), clone(t)
    for kw in (dict(step=0), dict(step=1, beta1=1.0), dict(step=1, beta2=-0.5), dict(step=1, eps=-1.0),
               dict(step=1, lr=float("nan")), dict(step=torch.ones(2, dtype=torch.int64, device="cuda")),
               dict(step=torch.ones(1, dtype=torch.int32, device="cuda")),
               dict(step=1, lr=torch.ones(1)), dict(step=1, grad_scale=2.0)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            L.adamw_step(plan, **{**HYPER, **kw})
    with pytest.raises(ValueError):
        L.adamw_state_values(plan)
    torch.cuda.synchronize()
    for k in t:
        assert all(torch.equal(a, b) for a, b in zip(t[k], old[k]))


def test_no_plan_inside_a_capture():
    L = ops()
    t = tensors([300], F32, F32, 32)
    L.adamw_step(L.adamw_plan(**t), 1, **HYPER)
    x = torch.zeros(4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x += 1
        with pytest.raises(RuntimeError):
            L.adamw_plan(**t)
    graph.replay()
    torch.cuda.synchronize()
    assert (x == 1).all()
