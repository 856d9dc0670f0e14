"""64-bit references of the 8-bit products and of the few-token layer, and the
bounds their tests use.  Written from the formulas, in float64 on the device
that holds the inputs."""
import torch

EPS32 = 2.0 ** -24                      # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def codes64(x):
    """round(127 x / max|x|) per row (exact: a tie's quotient is exact in
    float64) and max|x| / 127."""
    x = x.double()
    m = x.abs().amax(-1, keepdim=True)
    q = torch.round(127.0 * x / torch.where(m > 0, m, torch.ones_like(m)))
    return q, m[..., 0] / 127.0


def padded(q):
    """int8 codes with rows padded by zeros to a multiple of 128."""
    kp = (q.shape[-1] + 127) // 128 * 128
    out = torch.zeros((*q.shape[:-1], kp), dtype=torch.int8, device=q.device)
    out[..., :q.shape[-1]] = q.to(torch.int8)
    return out


def silu64(g):
    return g * torch.sigmoid(g)


def swiglu_error(g, u, eg, eu):
    """Bound on the error of fp32 silu(g) * u whose inputs are off by eg, eu:
    |silu'| <= 1.1, |silu| <= |g|; the exponential, sum, quotient and product
    round, and the exponential's argument error enters by |g|: 2^-20 covers
    (8 + |g|) 2^-24 for |g| <= 8 and silu's own size beyond it."""
    h = silu64(g) * u
    return 1.1 * eg * (u.abs() + eu) + g.abs() * eu + 2.0 ** -20 * (1 + g.abs()) * h.abs()


def mul8(q, s, w, t):
    """s t (q . w) and the bound of its fp32 scaling (conversion, scale product,
    product)."""
    y = (q.double() @ w.double().t()) * s[:, None].double() * t[None].double()
    return y, 4 * EPS32 * y.abs()


def expert8(x, gate, up, down):
    """One expert with 8-bit weights (pairs of codes and scales): y and a bound
    on the error of fp32 arithmetic around the exact integer sums.  A code of h
    may differ by one where h lies within its error of a rounding border."""
    q, s = codes64(x)
    g, eg = mul8(q, s, *gate)
    u, eu = mul8(q, s, *up)
    h = silu64(g) * u
    eh = swiglu_error(g, u, eg, eu)
    qh, sh = codes64(h)
    m = h.abs().amax(-1, keepdim=True)
    t = 127.0 * h / torch.where(m > 0, m, torch.ones_like(m))
    # error of the quotient: h's own and that of the row's maximum
    em = torch.where(h.abs() == m, eh, torch.zeros_like(eh)).amax(-1, keepdim=True)
    et = 127.0 * (eh + h.abs() / m.clamp_min(1e-300) * em) / m.clamp_min(1e-300)
    near = ((t.abs() - torch.floor(t.abs()) - 0.5).abs() <= et).double()
    y, ey = mul8(qh, sh, *down)
    w, td = down
    step = (near @ w.double().abs().t()) * sh[:, None] * td[None].double()
    rel_s = em / m.clamp_min(1e-300)
    return y, ey + step + rel_s * y.abs()


def expert_float(x, wg, wu, wd, h_rel):
    """One expert in float64 and the bound of fp32 sums of its K terms in any
    order; h_rel is the relative rounding of h before the down product."""
    x, wg, wu, wd = (v.double() for v in (x, wg, wu, wd))
    g, u = x @ wg.t(), x @ wu.t()
    a = x.shape[1] * EPS32
    eg, eu = a * (x.abs() @ wg.abs().t()), a * (x.abs() @ wu.abs().t())
    h = silu64(g) * u
    eh = swiglu_error(g, u, eg, eu) + h_rel * h.abs()
    y = h @ wd.t()
    ey = eh @ wd.abs().t() + wd.shape[1] * EPS32 * (h.abs() @ wd.abs().t())
    return y, ey


def route64(x, w_router, bias, S, gate_norm="ratio", gate_scale=1.0, k=6):
    z = x.double() @ w_router.double().t()
    E = z.shape[1] - S
    a = torch.sigmoid(z)
    idx = torch.sort(a[:, :E] + bias.double(), dim=1, descending=True,
                     stable=True).indices[:, :k]
    if gate_norm == "logsumexp":
        l = torch.nn.functional.logsigmoid(z)
        l = torch.cat([torch.gather(l, 1, idx), l[:, E:]], 1)
        g = torch.softmax(l, 1)
    else:
        s = torch.cat([torch.gather(a, 1, idx), a[:, E:]], 1)
        g = s / s.sum(1, keepdim=True)
    return idx, g * gate_scale


def layer64(x, idx, gates, expert, S):
    """Weighted sum of the experts' outputs for the picks idx; expert(kind, e, rows)
    returns (y, bound) of one expert on rows of x.  Returns y and its bound."""
    T, d = x.shape
    y = torch.zeros((T, d), dtype=torch.float64, device=x.device)
    b = torch.zeros_like(y)
    mag = torch.zeros_like(y)

    def add(rows, g, out):
        v, e = out
        y[rows] += g[:, None] * v
        b[rows] += g[:, None].abs() * e
        mag[rows] += (g[:, None] * v).abs()

    for e in torch.unique(idx).tolist():
        rows, slot = torch.nonzero(idx == e, as_tuple=True)
        add(rows, gates[rows, slot], expert("w", e, rows))
    every = torch.arange(T, device=x.device)
    for s in range(S):
        add(every, gates[:, idx.shape[1] + s], expert("ws", s, every))
    # gates rounded to fp32 and up to 48 fp32 additions of the weighted outputs
    return y, b + 50 * EPS32 * mag
