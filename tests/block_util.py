"""64-bit forms of the gated block, the e4m3 products and the AdamW step, with
bounds of what fp32 sums and the stated roundings may differ from them."""
import numpy as np
import torch

U32 = 2.0 ** -24                # half a step of fp32, relative
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def rand(shape, dtype, seed, scale=1.0, device="cuda", skew=0):
    """N(0, scale^2); with ``skew`` a dense tensor that starts `skew` values into its
    buffer."""
    g = torch.Generator().manual_seed(seed)
    n = 1
    for s in shape:
        n *= s
    flat = (torch.randn(n + skew, generator=g) * scale).to(dtype).to(device)
    return flat[skew:].view(shape)


def spans(offsets, M, E):
    """Row range of each group: offsets clamped to [0, M], none below one before it."""
    if offsets is None:
        return [(0, M)]
    out, top = [], 0
    for e in range(E):
        lo = max(top, min(max(offsets[e], 0), M))
        hi = max(lo, min(max(offsets[e + 1], 0), M))
        out.append((lo, hi))
        top = lo
    return out


def gated64(x, wg, wu, offsets, dh=None):
    """{name: (value, bound)} in float64.  Bounds: a sum of n fp32 products is within
    n U32 of the sum of their magnitudes; |silu'| <= 1.1, |silu''| <= 0.5; exp, the
    quotient and the products around them some 12 U32 relative; da and du, and the
    results, half a step of the type."""
    dt = x.dtype
    M, d = x.shape
    E, F, _ = wg.shape
    step = STEP[dt]
    out = {"h": [torch.zeros(M, F, dtype=torch.float64), torch.zeros(M, F, dtype=torch.float64)]}
    if dh is not None:
        out["dx"] = [torch.zeros(M, d, dtype=torch.float64) for _ in range(2)]
        for n in ("dw_gate", "dw_up"):
            out[n] = [torch.zeros(E, F, d, dtype=torch.float64) for _ in range(2)]
    covered = torch.zeros(M, dtype=torch.bool)
    X, G, U = (t.cpu().double() for t in (x, wg, wu))
    for e, (lo, hi) in enumerate(spans(offsets, M, E)):
        covered[lo:hi] = True
        if lo == hi:
            continue
        xs = X[lo:hi]
        a, u = xs @ G[e].T, xs @ U[e].T
        ea, eu = ((d + 4) * U32 * (xs.abs() @ w[e].abs().T) for w in (G, U))
        s = torch.sigmoid(a)
        silu = a * s
        h = silu * u
        out["h"][0][lo:hi] = h
        eh = 1.1 * ea * u.abs() + (silu.abs() + 1.1 * ea) * eu + 12 * U32 * h.abs()
        out["h"][1][lo:hi] = eh + step * (h.abs() + eh) + 1e-38
        if dh is None:
            continue
        g = dh[lo:hi].cpu().double()
        slope = s * (1 + a * (1 - s))
        da, du = g * u * slope, g * silu
        # 1 + a (1 - s) cancels for negative a: its error is relative to its terms
        terms = s * (1 + (a * (1 - s)).abs())
        eda = g.abs() * (u.abs() * (0.5 * ea + 12 * U32 * terms) + (1.1 + 0.5 * ea) * eu) + 1e-38
        edu = g.abs() * (1.1 * ea + 12 * U32 * silu.abs()) + 1e-38
        if dt == torch.bfloat16:
            eda, edu = eda + step * (da.abs() + eda), edu + step * (du.abs() + edu)
        dx = da @ G[e] + du @ U[e]
        edx = (eda + (2 * F + 4) * U32 * da.abs()) @ G[e].abs() + \
            (edu + (2 * F + 4) * U32 * du.abs()) @ U[e].abs()
        out["dx"][0][lo:hi], out["dx"][1][lo:hi] = dx, edx + step * (dx.abs() + edx) + 1e-38
        n = hi - lo
        for name, v, ev in (("dw_gate", da, eda), ("dw_up", du, edu)):
            w = v.T @ xs
            ew = (ev + (n + 4) * U32 * v.abs()).T @ xs.abs()
            out[name][0][e], out[name][1][e] = w, ew + step * (w.abs() + ew) + 1e-38
    return {n: tuple(v) for n, v in out.items()}, covered


def within(got, want, bound, what=""):
    """Every value of got within its bound of want."""
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
        f"{float((off / bound.clamp(min=1e-300)).max()):.3g} times the bound")


# ------------------------------------------------------------------- e4m3

E4M3 = torch.tensor(sorted({(8 + f) * 2.0 ** (e - 10) for e in range(1, 16) for f in range(8)} |
                           {f * 2.0 ** -9 for f in range(8)})[:-1], dtype=torch.float64)


def e4m3_codes(t):
    """Codes (uint8) of the e4m3 values nearest to t (float64), ties to the even code."""
    mag = t.abs().contiguous()
    hi = torch.searchsorted(E4M3, mag).clamp(1, len(E4M3) - 1)
    down, up = mag - E4M3[hi - 1], E4M3[hi] - mag
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    return (code + 128 * torch.signbit(t)).to(torch.uint8)


def scale_of(top):
    """fp32 scale (as float64) of blocks of largest magnitude `top` (float64)."""
    s = (top / 448.0).float().clamp(min=2.0 ** -126).double()
    return torch.where(top > 0, s, torch.zeros_like(s))


def quantise64(x):
    """Codes [rows, Kp] (uint8) and scales [rows, Kp/128] (float64) of fp32 or bf16 x."""
    x = x.cpu().double()
    rows, K = x.shape
    b = (K + 127) // 128
    x = torch.nn.functional.pad(x, (0, b * 128 - K)).view(rows, b, 128)
    bad = ~torch.isfinite(x).all(-1)
    s = scale_of(torch.where(bad[..., None], torch.zeros_like(x), x).abs().amax(-1))
    q = x / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    codes = e4m3_codes(torch.where(bad[..., None], torch.zeros_like(q), q))
    codes[bad | (s == 0)] = 0
    return codes.view(rows, -1), torch.where(bad, torch.full_like(s, float("nan")), s)


def fp8_product64(a, a_scale, w, w_scale, offsets, out_dtype):
    """(value, bound, covered rows) of the product of codes."""
    A = a.cpu().double() * a_scale.cpu().double().repeat_interleave(128, 1)
    E, N, Kp = w.shape
    W = w.cpu().double() * w_scale.cpu().double().repeat_interleave(128, 1)[:, :N] \
        .repeat_interleave(128, 2)
    M = A.shape[0]
    y, b = (torch.zeros(M, N, dtype=torch.float64) for _ in range(2))
    covered = torch.zeros(M, dtype=torch.bool)
    for e, (lo, hi) in enumerate(spans(offsets, M, E)):
        covered[lo:hi] = True
        y[lo:hi] = A[lo:hi] @ W[e].T
        # products of codes are exact; each addition may be off by a step (2 U32) of
        # the sum of magnitudes, the scales' product and its use by one more each
        b[lo:hi] = (Kp + 4) * 2 * U32 * (A[lo:hi].abs() @ W[e].abs().T)
    return y, b + STEP[out_dtype] * (y.abs() + b) + 1e-38, covered


# ------------------------------------------------------------------ AdamW

def adamw64(p, g, m, v, step, lr, b1, b2, eps, wd, factor, ms=None, vs=None):
    """One step in float64; 8-bit states with scales ms, vs give codes and scales."""
    P, Gr = p.cpu().double(), g.cpu().double() * factor
    M, V = m.cpu().double(), v.cpu().double()
    if ms is not None:
        rep = lambda s: s.cpu().double().repeat_interleave(256)[:M.numel()].view(M.shape)
        M = rep(ms) * M * M.abs() / 127.0 ** 2
        V = rep(vs) * V ** 4 / 255.0 ** 4
    new_m = b1 * M + (1 - b1) * Gr
    new_v = b2 * V + (1 - b2) * Gr ** 2
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    den = torch.sqrt(new_v / c2) + eps
    upd = lr * (new_m / c1) / den
    out = {"p": P * (1 - lr * wd) - upd, "m": new_m, "v": new_v}
    # m': two products and a sum of rounded constants, 4 U32 of the terms; v': 6 U32
    # relative; p': m's error over the root, and some 16 roundings of the update
    em = 4 * U32 * ((b1 * M).abs() + ((1 - b1) * Gr).abs()) + 1e-44
    out["em"], out["ev"] = em, 6 * U32 * new_v + 1e-44
    # (magnitudes: lr may be negative)
    out["ep"] = abs(lr) / c1 * em / den + 16 * U32 * upd.abs() + 3 * U32 * P.abs() + 1e-44
    if ms is not None:
        n = M.numel()
        pad = (n + 255) // 256 * 256 - n
        bm = torch.nn.functional.pad(new_m.flatten(), (0, pad)).view(-1, 256)
        bv = torch.nn.functional.pad(new_v.flatten(), (0, pad)).view(-1, 256)
        s, z = bm.abs().amax(1).float(), bv.amax(1).float()
        safe = lambda t: torch.where(t > 0, t, torch.ones_like(t)).double()[:, None]
        # roots in 64-bit mantissas: a quarter of the largest lies on a border (127 / 2 =
        # 63.5), and bf16 gradients meet it, often one step of 64 bits (2^-52) below.
        # The root halves that to 2^-53, which a root in 53 bits rounds away.
        wide = lambda t: t.numpy().astype(np.longdouble)
        narrow = lambda a: torch.from_numpy(np.rint(a).astype(np.float64))
        cm = torch.sign(bm) * narrow(127 * np.sqrt(wide(bm.abs()) / wide(safe(s)))).clamp(max=127)
        cv = narrow(255 * np.sqrt(np.sqrt(wide(bv) / wide(safe(z))))).clamp(max=255)
        cv = torch.where(bv > 0, cv.clamp(min=1), cv)
        out.update(cm=cm.flatten()[:n].view(M.shape).to(torch.int8),
                   cv=cv.flatten()[:n].view(M.shape).to(torch.uint8), s=s, z=z)
    return out
