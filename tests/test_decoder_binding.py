"""The binding's side of the decoder-step calls, without a GPU: what the
allocator is told, what is refused, what a step's status says."""
from types import SimpleNamespace

import pytest


@pytest.fixture(scope="module")
def S():
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


class _Told:
    """A tensor that keeps what its allocator was told, and when."""

    def __init__(self, log):
        self.log = log

    def record_stream(self, stream):
        self.log.append((self, stream))


@pytest.mark.parametrize("scales", [True, False])
@pytest.mark.parametrize("call", ["kv_write", "kv_read", "attn_decode"])
def test_a_given_stream_is_told_of_the_cache(S, monkeypatch, call, scales):
    log = []
    tensors = [_Told(log) for _ in range(4 if scales else 2)]
    cache = SimpleNamespace(address=1, index=0, **dict(zip(("k", "v", "k_scales", "v_scales"), tensors + [None, None])))
    native = SimpleNamespace(**{call: lambda *a: log.append("called") or "out"})
    monkeypatch.setattr(S, "_bind", native)
    args = {"kv_write": (cache, "k", "v", "slots", "ws"), "kv_read": (cache, "slots", "ws"),
            "attn_decode": ("q", cache, "table", "lens", "ws")}[call]
    assert getattr(S, call)(*args) == (None if call == "kv_write" else "out")
    assert log == ["called"]                       # the current stream needs no word
    log.clear()
    getattr(S, call)(*args, stream="side")
    assert log == ["called"] + [(t, "side") for t in tensors]


@pytest.mark.parametrize("linears,attention,first", [(6, 7, 6), (0, 7, 7), (6, 0, 6), (0, 0, 0)])
def test_status_reads_and_clears_both_workspaces(S, monkeypatch, linears, attention, first):
    from w4_gemm_gated_b200 import decoder
    words = {"ws": linears, "attn_ws": attention}

    def read_status(ws):
        word, words[ws] = words[ws], 0
        return word

    monkeypatch.setattr(decoder, "S", SimpleNamespace(read_status=read_status))
    state = SimpleNamespace(ws="ws", attn_ws="attn_ws")
    assert decoder.status(state) == first
    assert words == {"ws": 0, "attn_ws": 0} and decoder.status(state) == 0
