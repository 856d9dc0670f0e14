"""What the binding of the gated block, the e4m3 products and the AdamW step does on
the host (no GPU: streams, tables and launches are stand-ins)."""
import contextlib

import pytest
import torch

L = pytest.importorskip("sparse_mixture_experts_04_amd._lib")


class Table:
    """A plan's table that notes the streams it is told of."""

    def __init__(self):
        self.streams = []

    def data_ptr(self):
        return 0x1000

    def record_stream(self, stream):
        self.streams.append(stream)


@pytest.fixture
def host(monkeypatch):
    """No GPU: calls succeed, the current stream's handle is host["stream"]."""
    state = {"stream": 0, "capturing": False, "calls": []}
    monkeypatch.setattr(L, "_raw_stream", lambda idx: state["stream"])
    monkeypatch.setattr(L, "_call", lambda idx, fn, *args: state["calls"].append(fn) or 0)
    monkeypatch.setattr(torch.cuda, "device", lambda idx: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("stream", state["stream"]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    return state


def plan():
    p = L.AdamwPlan.__new__(L.AdamwPlan)
    p.device, p.desc, p.chunks, p.table = 0, L.AdamwDesc(1, L.F32, L.F32, 8), 1, Table()
    p.tensors, p.stream = {"m_values": [None]}, 7
    return p


def test_a_plans_table_is_kept_for_steps_on_other_streams(host):
    """torch may give the memory of a dropped plan to the stream it was made on; a step
    on another one that still reads the table has to be known to torch."""
    p = plan()
    host["stream"] = 7  # the plan's own: memory freed on it is used again in its order
    L.adamw_step(p, 1, lr=1e-3)
    L.adamw_state_values(p)
    assert p.table.streams == [] and len(host["calls"]) == 2
    host["stream"] = 9
    L.adamw_step(p, 2, lr=1e-3)
    assert p.table.streams == [("stream", 9)]
    host["stream"] = 11
    L.adamw_state_values(p)
    assert p.table.streams == [("stream", 9), ("stream", 11)]


def test_a_captured_step_leaves_the_plan_to_the_graphs_owner(host):
    p = plan()
    host.update(stream=9, capturing=True)
    L.adamw_step(p, 1, lr=1e-3)
    assert p.table.streams == [] and len(host["calls"]) == 1


WIDE = (1 << 32) + 128  # its low 32 bits are a size that calls take


@pytest.mark.parametrize("make", [
    lambda n: L.GatedFfDesc(1, n, 8, 1, L.BF16), lambda n: L.GatedFfDesc(n, 8, 8, 1, L.BF16),
    lambda n: L.GatedFfDesc(1, 8, F=n, E=1), lambda n: L.GatedFfDesc(1, 8, 8, n),
    lambda n: L.GemmFp8Desc(1, n, 128, 1, L.BF16), lambda n: L.GemmFp8Desc(M=1, N=8, K=n, E=1, out=L.F32),
    lambda n: L.GemmInt8Desc(n, 8, 128, 1, L.BF16), lambda n: L.GemmInt8Desc(1, 8, 128, n, L.BF16),
    lambda n: L.make_desc(n, 512, 128, torch.bfloat16), lambda n: L.make_desc(4, n, 128, torch.bfloat16),
    lambda n: L.Desc(T=4, d=512, F=n), lambda n: L.make_desc(4, 512, 128, torch.bfloat16, k=n),
    lambda n: L.gated_ff_workspace(n, 8, 8, 1, torch.bfloat16, "cpu"),
    lambda n: L.gated_ff_workspace(1, 8, n, 1, torch.bfloat16, "cpu"),
    lambda n: L.gemm_fp8_workspace(1, 8, n, device="cpu"),
    lambda n: L.gemm_int8_workspace(1, n, 128, device="cpu"),
])
@pytest.mark.parametrize("n", [WIDE, 1 << 31, -WIDE, (1 << 63) + 8])
def test_sizes_of_more_than_32_bits_are_refused(make, n):
    """They are not cut to their low 32 bits."""
    with pytest.raises(L.MoEError) as e:
        make(n)
    assert e.value.status == 5


@pytest.mark.parametrize("call,shape", [
    (lambda x: L.quantize_fp8(x), (0, WIDE)), (lambda x: L.quantize_int8(x), (0, WIDE)),
    (lambda x: L.quantize_fp8_weights(x), (0, 8, WIDE)), (lambda x: L.quantize_fp8_weights(x), (0, WIDE, 8)),
    (lambda x: L.quantize_fp8_weights(x), (WIDE, 0, 8)), (lambda x: L.quantize_mxfp4(x), (0, 8, WIDE)),
])
def test_rows_of_more_than_32_bits_are_refused(monkeypatch, call, shape):
    """Of tensors too: the library would see a row of 128 values (no values here, so
    that nothing is launched)."""
    monkeypatch.setattr(L, "_on_gpu", lambda x, name: 0)
    monkeypatch.setattr(L, "_at", lambda *a: 0x1000)
    monkeypatch.setattr(L, "_ptr", lambda *a: 0x1000)
    monkeypatch.setattr(L, "_stream", lambda d: None)
    monkeypatch.setattr(L, "_call", lambda idx, fn, *args: fn(*args, None))
    with pytest.raises(L.MoEError) as e:
        call(torch.empty(shape, dtype=torch.bfloat16, device="meta"))
    assert e.value.status == 5


def test_sizes_of_32_bits_keep_their_meaning():
    d = L.GatedFfDesc(1, 2, 3, 4, L.BF16)
    assert (d.M, d.d, d.F, d.E, d.act) == (1, 2, 3, 4, L.BF16)
    d = L.GemmFp8Desc(-1, 5, out=L.BF16, K=(1 << 31) - 1)
    assert (d.M, d.N, d.K, d.E, d.out) == (-1, 5, (1 << 31) - 1, 0, L.BF16)
    d = L.make_desc(8, 512, 128, torch.bfloat16, E=64, S=1, k=4, gate_norm="logsumexp", gate_scale=2.5,
                    capacity_factor=1.25)
    assert (d.T, d.d, d.F, d.E, d.S, d.k) == (8, 512, 128, 64, 1, 4)
    assert (d.act, d.weight, d.gate_norm, d.gate_scale, d.capacity_factor) == (
        L.BF16, L.BF16, L.GATE_LOGSUMEXP, 2.5, 1.25)


def test_steps_of_more_than_64_bits_are_refused(host):
    for step in (1 << 63, (1 << 64) + 5):
        with pytest.raises(ValueError):
            L.adamw_step(plan(), step, lr=1e-3)
    assert not host["calls"]


@pytest.mark.parametrize("current,captured,refused", [(0, 1, True), (0, 0, True), (0, None, False),
                                                      (1, 1, True), (1, None, False)])
def test_no_plan_where_either_gpus_stream_is_captured(monkeypatch, host, current, captured, refused):
    """Of the current GPU or of the tensors' own (cuda:1 here): the table's kernels would
    go into the capture, and the wait behind them would end it."""
    at = [current]

    @contextlib.contextmanager
    def device(idx):
        before, at[0] = at[0], idx
        yield
        at[0] = before

    class Stream:
        def synchronize(self):
            host["calls"].append("wait")

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: at[0] == captured)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(L, "_on_gpu", lambda x, name: 1)
    monkeypatch.setattr(L, "_at", lambda *a: 0x1000)
    x = torch.zeros(4)
    if refused:
        with pytest.raises(RuntimeError, match="before the capture"):
            L.adamw_plan([x], [x], [x], [x])
        assert host["calls"] == []
    else:
        assert L.adamw_plan([x], [x], [x], [x]).device == 1
        assert host["calls"][-1] == "wait"
    assert at[0] == current
