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
