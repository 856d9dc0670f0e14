"""The e4m3 quantisers and products against their definition in 64 bits."""
import pytest
import torch

from block_util import E4M3, fp8_product64, quantise64, rand, scale_of, e4m3_codes, within

pytestmark = pytest.mark.gpu
BF, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def ops():
    from sparse_mixture_experts_04_amd import ops
    return ops


def same_codes(got, want):
    """Equal codes; a zero's sign does not matter."""
    g = got.cpu().view(torch.uint8)
    ok = (g == want) | ((g & 0x7f == 0) & (want & 0x7f == 0))
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()} codes differ"


def check_rows(x):
    codes, scales = ops().quantize_fp8(x)
    q, s = quantise64(x)
    assert torch.equal(torch.nan_to_num(scales.cpu().double(), -1.0), torch.nan_to_num(s, -1.0))
    same_codes(codes, q)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 8), (2, 127), (5, 128), (7, 129), (16, 300), (33, 1111),
                                    (200, 2048), (65, 7168), (1, 4096), (1000, 72)])
def test_quantize_rows(rows, K, dt):
    x = rand((rows, K), dt, rows + K) * torch.exp2(torch.arange(rows, device="cuda") % 40 - 20.0)[:, None]
    check_rows(x.to(dt))


@pytest.mark.parametrize("skew", [1, 3, 4])
def test_quantize_unaligned(skew):
    for dt in (BF, F32):
        check_rows(rand((9, 260), dt, 1, skew=skew))


def test_quantize_borders():
    """Values at every border between two codes, and one step of fp32 to either side,
    in blocks whose scale is no power of two."""
    mids = (E4M3[1:] + E4M3[:-1]) / 2
    for top in (1.0, 0.7, 3.1e-3, 5e20, 448.0):
        s = scale_of(torch.tensor(top, dtype=torch.float32).double())
        v = (mids * s).float()
        v = torch.cat([v, torch.nextafter(v, torch.tensor(0.0)), torch.nextafter(v, torch.tensor(9e37))])
        v = torch.cat([v, -v])
        n = (v.numel() + 126) // 127
        x = torch.zeros(n, 128)
        x[:, 0] = top
        x[:, 1:].reshape(-1)  # (a view keeps the first column)
        flat = torch.zeros(n * 127)
        flat[:v.numel()] = v
        x[:, 1:] = flat.view(n, 127)
        check_rows(x.cuda())


def test_quantize_extremes():
    x = torch.zeros(8, 256)
    x[0, :128] = 1e-45 * torch.arange(128)          # the smallest numbers there are
    x[1] = 3.4e38
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4, 7] = -1e-37
    x[5] = torch.linspace(-1, 1, 256) * 2e-36
    x[6, 0], x[6, 1] = 1.0, 1e-30
    check_rows(x.cuda())


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (2, 130, 129), (3, 128, 256), (1, 300, 72), (5, 7, 1000)])
def test_quantize_weights(E, N, K, dt):
    w = rand((E, N, K), dt, N + K)
    w[0, 0] *= 50
    if E > 1:
        w[1, :, :] = 0
    codes, scales = ops().quantize_fp8_weights(w)
    nb, kb = (N + 127) // 128, (K + 127) // 128
    big = torch.zeros(E, nb * 128, kb * 128, dtype=torch.float64)
    big[:, :N, :K] = w.cpu().double()
    blocks = big.view(E, nb, 128, kb, 128)
    s = scale_of(blocks.abs().amax((2, 4)))
    assert torch.equal(scales.cpu().double(), s)
    q = blocks / torch.where(s > 0, s, torch.ones_like(s))[:, :, None, :, None]
    same_codes(codes, e4m3_codes(q).view(E, nb * 128, kb * 128)[:, :N])


def test_quantize_weights_with_nan():
    w = rand((1, 200, 200), F32, 3)
    w[0, 150, 20] = float("nan")
    codes, scales = ops().quantize_fp8_weights(w)
    assert torch.isnan(scales).sum() == 1 and torch.isnan(scales[0, 1, 0])
    assert not codes.view(torch.uint8)[0, 128:, :128].any()


def operands(M, N, K, E, seed=0):
    L = ops()
    a, sa = L.quantize_fp8(rand((M, K), F32, seed + 1))
    w, sw = L.quantize_fp8_weights(rand((E, N, K), F32, seed + 2, K ** -0.5))
    return a, sa, w, sw


def check_product(M, N, K, offsets=None, dt=F32, seed=0, ops_=None):
    L = ops()
    E = 1 if offsets is None else len(offsets) - 1
    a, sa, w, sw = operands(M, N, K, E, seed) if ops_ is None else ops_
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = torch.full((M, N), 7.0, dtype=dt, device="cuda")
    ws = L.gemm_fp8_workspace(M, N, K, E)
    ws.fill_(0xff)
    L.gemm_fp8(a, sa, w, sw, y, offsets=off, ws=ws)
    want, bound, covered = fp8_product64(a, sa, w, sw, offsets, dt)
    within(y[covered.cuda()], want[covered], bound[covered])
    assert (y.cpu()[~covered] == 7.0).all()
    return y


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 128), (1, 2048, 7168), (2, 130, 300), (7, 129, 1000),
                                   (16, 768, 2048), (17, 100, 128), (33, 257, 384), (100, 770, 1111),
                                   (128, 256, 128), (129, 255, 640), (300, 520, 256), (1100, 300, 512),
                                   (2050, 1300, 128)])
def test_product(M, N, K, dt):
    check_product(M, N, K, dt=dt, seed=M + N)


@pytest.mark.parametrize("M,N,K,offsets", [
    (40, 64, 256, [0, 40]),
    (40, 100, 200, [0, 0, 13, 13, 40, 40]),
    (64, 272, 72, [3, 20, 20, 50]),
    (50, 128, 140, [0, 70, 60, -5, 50]),
    (9, 140, 384, [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]),
    (900, 512, 136, [0, 257, 258, 300, 555, 900]),
    (3000, 256, 256, [0, 1, 129, 385, 1386, 3000]),
])
def test_groups(M, N, K, offsets):
    check_product(M, N, K, offsets, dt=BF)
    check_product(M, N, K, offsets, dt=F32)


@pytest.mark.parametrize("per", [1, 6, 20, 90])
def test_256_groups(per):
    g = torch.Generator().manual_seed(per)
    n = torch.randint(0, 2 * per + 1, (256,), generator=g)
    off = [0] + torch.cumsum(n, 0).tolist()
    check_product(max(off[-1], 1), 136, 256, off, dt=BF)


def test_scales_that_differ_widely():
    """Blocks of K whose scales lie 2^30 apart, and a weight block of scale 0."""
    a, sa, w, sw = operands(40, 300, 640, 1)
    sa = sa * torch.exp2(torch.tensor([0.0, 30, -30, 10, -20], device="cuda"))[None]
    sw = sw * torch.exp2(torch.tensor([5.0, -25, 20, 0, 10], device="cuda"))[None, None]
    sw[0, 1, 2] = 0
    check_product(40, 300, 640, ops_=(a, sa.contiguous(), w, sw.contiguous()))


def test_every_code_value():
    """All 254 finite codes against a row of ones."""
    L = ops()
    codes = torch.tensor([c for c in range(256) if c & 0x7f != 0x7f], dtype=torch.uint8, device="cuda")
    a = torch.zeros((254, 128), dtype=torch.uint8, device="cuda")
    a[:, 77] = codes
    w = torch.ones((1, 130, 128), device="cuda").to(FP8)
    one = torch.ones((254, 1), device="cuda")
    y = torch.empty((254, 130), device="cuda")
    L.gemm_fp8(a.view(FP8), one, w, torch.ones((1, 2, 1), device="cuda"), y)
    assert torch.equal(y, codes.view(FP8).float()[:, None].expand(254, 130))


@pytest.mark.parametrize("M", [3, 200, 700])
def test_nan_stays_in_its_row_and_column(M):
    a, sa, w, sw = operands(M, 300, 256, 1)
    clean = check_product(M, 300, 256, ops_=(a, sa, w, sw))
    sa = sa.clone()
    sa[1, 1] = float("nan")
    sw = sw.clone()
    sw[0, 2, 0] = float("nan")
    y = torch.empty_like(clean)
    ops().gemm_fp8(a, sa, w, sw, y)
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 256:]).all()
    keep = [r for r in range(M) if r != 1]
    assert torch.equal(y[keep, :256], clean[keep, :256])


def test_same_bits_again_and_captured():
    L = ops()
    a, sa, w, sw = operands(333, 500, 900, 3)
    off = torch.tensor([0, 100, 101, 333], dtype=torch.int32, device="cuda")
    y = [torch.empty((333, 500), dtype=BF, device="cuda") for _ in range(2)]
    ws = L.gemm_fp8_workspace(333, 500, 900, 3)
    L.gemm_fp8(a, sa, w, sw, y[0], offsets=off, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.gemm_fp8(a, sa, w, sw, y[1], offsets=off, ws=ws)
    s.synchronize()
    assert torch.equal(*y)
    graph = torch.cuda.CUDAGraph()
    x = rand((333, 900), BF, 1)
    a2, sa2 = torch.empty_like(a), torch.empty_like(sa)
    with torch.cuda.graph(graph):
        L.quantize_fp8(x, a2, sa2)
        L.gemm_fp8(a2, sa2, w, sw, y[1], offsets=off, ws=ws)
    for i in range(3):
        x.copy_(rand((333, 900), BF, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        c, sc = L.quantize_fp8(x)
        L.gemm_fp8(c, sc, w, sw, y[0], offsets=off)
        assert torch.equal(*y), i


def test_no_rows():
    L = ops()
    a, sa, w, sw = operands(1, 40, 128, 1)
    y = torch.empty((0, 40), device="cuda")
    L.gemm_fp8(a[:0], sa[:0], w, sw, y)
    c, s = L.quantize_fp8(torch.empty((0, 40), device="cuda"))
    assert c.shape == (0, 128) and s.shape == (0, 1)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,offsets", [(256, 520, [3, 200]), (256, 333, [0, 256]), (9, 130, [1, 9]),
                                         (8, 130, [2, 7]), (100, 2048, [50, 50]), (130, 258, None)])
def test_slices_of_k(M, N, offsets, dt):
    """One group of part of the rows, columns of any number."""
    check_product(M, N, 3500, offsets, dt=dt, seed=M + N)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,offsets", [
    (256, 2048, 3500, [3, 200]), (256, 1999, 3500, None), (700, 1030, 3500, [0, 699]),
    (1024, 2048, 7000, [3, 1000]), (1000, 1999, 7000, None), (1100, 2050, 7000, [50, 50])])
def test_slices_of_k_in_memory(M, N, K, offsets, dt):
    """A product whose tiles are cut along K, their sums in the workspace (the last
    three; smaller ones are not cut)."""
    assert M < 1000 or ops().gemm_fp8_workspace(M, N, K).numel() > 1
    check_product(M, N, K, offsets, dt=dt, seed=M + N)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,offsets", [(3, 5000, 3000, None), (8, 7168, 1920, [1, 8]),
                                           (5, 900, 5000, [0, 2, 2, 5])])
def test_few_rows_of_many_weights(M, N, K, offsets, dt):
    check_product(M, N, K, offsets, dt=dt, seed=M + N)


@pytest.mark.parametrize("M,N,K,offsets", [
    (4200, 3104, 256, None), (4100, 3100, 300, [2, 4099]),
    (6000, 2200, 640, [0, 1, 1, 2048, 2305, 5990]), (25000, 600, 128, None)])
def test_large_tiles(M, N, K, offsets):
    """256 x 256 tiles: last tiles that are not whole, groups that end inside one."""
    check_product(M, N, K, offsets, dt=BF, seed=M)


def test_two_products_at_once():
    L = ops()
    sets = [operands(256, 2048, 3584, 1, seed=s) for s in (1, 5)]
    want = [torch.empty((256, 2048), dtype=BF, device="cuda") for _ in sets]
    got = [torch.zeros_like(t) for t in want]
    for s, y in zip(sets, want):
        L.gemm_fp8(*s, y)
    wss = [L.gemm_fp8_workspace(256, 2048, 3584) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, y, ws, st in zip(sets, got, wss, streams):
            with torch.cuda.stream(st):
                L.gemm_fp8(*s, y, ws=ws)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_a_row_does_not_depend_on_the_batch_of_its_tile():
    """Rows of one group beside others of any values: same bits."""
    a, sa, w, sw = operands(300, 520, 640, 1)
    y = check_product(300, 520, 640, ops_=(a, sa, w, sw), dt=BF)
    a2, sa2 = a.clone(), sa.clone()
    a2.view(torch.uint8)[100:] = 0x7f          # NaN
    y2 = torch.empty_like(y)
    ops().gemm_fp8(a2, sa2, w, sw, y2)
    assert torch.equal(y[:100], y2[:100]) and torch.isnan(y2[100:]).all()


def test_refusals_of_the_binding():
    L = ops()
    a, sa, w, sw = operands(20, 40, 200, 2)
    off = torch.tensor([0, 9, 20], dtype=torch.int32, device="cuda")
    y = torch.zeros((20, 40), device="cuda")
    with pytest.raises(RuntimeError):
        L.gemm_fp8(a, sa, w, sw, y)                                # offsets missing
    for args in ((a.view(torch.uint8), sa, w, sw, y), (a[:, :128], sa, w, sw, y),
                 (a[:, :200], sa, w, sw, y), (a, sa[:, :1], w, sw, y), (a, sa.to(BF), w, sw, y),
                 (a, sa, w[:, :30], sw, y), (a, sa, w, sw[:, :, :1], y), (a, sa, w[0], sw, y),
                 (a, sa, w, sw, y[:10]), (a, sa, w, sw, y.half()), (a, sa, w, sw, y.t())):
        with pytest.raises((TypeError, ValueError)):
            L.gemm_fp8(*args, offsets=off)
    for x in (y.half(), y.long(), y.t(), torch.zeros((), device="cuda"), y[:, :0]):
        with pytest.raises((TypeError, ValueError)):
            L.quantize_fp8(x)
    with pytest.raises((TypeError, ValueError)):
        L.quantize_fp8(y, codes=torch.empty((20, 40), dtype=FP8, device="cuda"))
    with pytest.raises((TypeError, ValueError)):
        L.quantize_fp8_weights(y)
    flat = torch.zeros(20 * 128 + 8, dtype=torch.uint8, device="cuda")
    with pytest.raises(RuntimeError):                              # codes not on 16 bytes
        L.quantize_fp8(y, codes=flat[8:].view(20, 128).view(FP8))
    torch.cuda.synchronize()
    assert not y.any() and not flat.any()
