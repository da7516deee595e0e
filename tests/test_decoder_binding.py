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


def _attn(S, **kw):
    """spear_attn_decode with a workspace that is too small: 4 once all else is in order."""
    import ctypes
    d = dict(q=0x100000, out=0x200000, ld=4096, seqs=3, table=0x300000, ld_table=6, lens=0x400000, lse=0x500000)
    d.update(kw)
    cache = S.KVCacheStruct(kind=1, n_pages=10, page_size=16, n_heads=8, head_dim=128, k=0x1000000, v=0x2000000,
                            k_scales=0x3000000, v_scales=0x4000000)
    return S.F["spear_attn_decode"](ctypes.byref(cache), d["q"], d["ld"], d["seqs"], 32, d["table"], 4, d["ld_table"],
                                    d["lens"], 0.1, d["out"], d["ld"], d["lse"], 0x600000, 255, None)


ROWS = 3 * 4096 * 2      # bytes of q and out
LSE = 3 * 32 * 4


@pytest.mark.parametrize("kw", [
    dict(lse=0x100000), dict(lse=0x100000 + ROWS - 4), dict(lse=0x100000 - LSE + 4),       # q's rows
    dict(lse=0x200000 + 8192), dict(lse=0x200000 - LSE + 4),                               # out's
    dict(lse=0x400000), dict(lse=0x400000 + 8), dict(lse=0x300000 + 4 * 15), dict(lse=0x300000 - LSE + 4),
    dict(lens=0x200000), dict(table=0x200000 + ROWS - 16), dict(table=0x200000 - 4 * 16 + 4),
])
def test_attn_refuses_outputs_over_its_inputs(S, kw):
    assert _attn(S, **kw) == S.ERR_INVALID_ARG and "overlap" in S.F["spear_last_error"]().decode()


@pytest.mark.parametrize("kw", [
    {}, dict(lse=None), dict(lse=0x100000 + ROWS), dict(lse=0x200000 - LSE), dict(lse=0x400000 + 12),
    dict(lse=0x400000 - LSE), dict(lse=0x300000 + 4 * 16), dict(table=0x200000 + ROWS), dict(lens=0x200000 - 12),
])
def test_attn_takes_outputs_beside_its_inputs(S, kw):
    assert _attn(S, **kw) == S.ERR_WORKSPACE


@pytest.mark.parametrize("scale,code", [(2.3e38, 4), (-2.3e38, 4), (2.4e38, 1), (-3.4e38, 1)])
def test_attn_refuses_a_scale_past_its_range_in_powers_of_two(S, scale, code):
    # scores are taken in powers of two: scale times log2(e) has to be finite too
    import ctypes
    cache = S.KVCacheStruct(kind=0, n_pages=10, page_size=16, n_heads=8, head_dim=128, k=0x1000000, v=0x2000000)
    assert S.F["spear_attn_decode"](ctypes.byref(cache), 0x100000, 4096, 3, 32, 0x300000, 4, 4, 0x400000, scale, 0x200000,
                                    4096, None, 0x600000, 255, None) == code


def _child(tmp_path, code):
    import os
    import subprocess
    import sys

    from tests.conftest import ROOT
    # the package with everything built but the native module
    pkg = tmp_path / "w4_gemm_gated_b200"
    pkg.mkdir()
    src = os.path.join(ROOT, "w4_gemm_gated_b200")
    for name in os.listdir(src):
        if not name.startswith("_bind") and name != "__pycache__":
            os.symlink(os.path.join(src, name), pkg / name)
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                          env=dict(os.environ, PYTHONPATH=str(tmp_path)))


def test_the_layer_calls_need_no_native_module(S, tmp_path):
    res = _child(tmp_path, "from w4_gemm_gated_b200 import spear as S, decoder\n"
                           "assert S.F['spear_device_checks_enabled']() == 0\n"
                           "print(S.LIB_PATH)")
    assert res.returncode == 0, res.stderr
    assert str(tmp_path) in res.stdout


@pytest.mark.parametrize("call", ["S.block_norm(None)", "S.kv_read(c, None, None)", "S.kv_write(c, 0, 0, 0, 0)",
                                  "S.attn_decode(0, c, 0, 0, 0)"])
def test_the_others_name_the_command_that_builds_it(S, tmp_path, call):
    res = _child(tmp_path, "from types import SimpleNamespace\nfrom w4_gemm_gated_b200 import spear as S\n"
                           f"c = SimpleNamespace(address=1, index=0)\ntry:\n    {call}\nexcept ImportError as e:\n    print(e)")
    assert res.returncode == 0, res.stderr
    assert "_bind" in res.stdout and "python -m w4_gemm_gated_b200.build" in res.stdout


def test_the_native_module_is_rebuilt_for_another_torch(S, monkeypatch, tmp_path):
    from w4_gemm_gated_b200 import build
    built = []
    monkeypatch.setattr(build.subprocess, "run",
                        lambda cmd, **kw: built.append(cmd) or SimpleNamespace(returncode=0, stdout="", stderr=""))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    versions = ["1.0+a"]
    monkeypatch.setattr(build, "torch_version", lambda: versions[0])
    build.build_bind()
    assert len(built) == 1                      # nothing says which torch the one there is of
    build.build_bind()
    assert len(built) == 1
    versions[0] = "1.0+b"
    build.build_bind()
    assert len(built) == 2
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: SimpleNamespace(returncode=1, stdout="", stderr="no"))
    versions[0] = "1.1"
    for _ in range(2):                          # a build that failed leaves no mark
        with pytest.raises(RuntimeError):
            build.build_bind()


PAGE = 8 * 16 * 128          # bytes of a page of int8 keys
PAGE_SCALES = 8 * 16 * 2


def _write(S, **kw):
    """spear_kv_write of too many tokens: unsupported (2) once the cache is in order."""
    import ctypes
    d = dict(kind=1, n_pages=10, page_size=16, n_heads=8, head_dim=128, k=0x1000000, v=0x2000000, k_scales=0x3000000,
             v_scales=0x4000000)
    d.update(kw)
    return S.F["spear_kv_write"](ctypes.byref(S.KVCacheStruct(**d)), 0x100000, 1024, 0x200000, 1024, 0x300000,
                                 2147483647, 0x400000, 256, None)


@pytest.mark.parametrize("kw", [
    dict(v=0x1000000), dict(v=0x1000000 + 16), dict(v=0x1000000 + 10 * PAGE - 16), dict(v=0x1000000 - 10 * PAGE + 16),
    dict(v=0x1000000, n_pages=1), dict(k_scales=0x4000000), dict(v_scales=0x3000000 + PAGE_SCALES),
    dict(page_stride=2 * PAGE, v=0x1000000 + PAGE - 16), dict(page_stride=2 * PAGE, v=0x1000000 + PAGE + 16),
    dict(page_stride=2 * PAGE - 16, v=0x1000000 + PAGE), dict(page_stride=2 * PAGE, v=0x1000000 + 4 * PAGE),
    dict(kind=0, k_scales=None, v_scales=None, v=0x1000000 + 2 * PAGE),
    # scales in the pages' rows: of the keys over the values
    dict(page_stride=4 * PAGE, scale_stride=2 * PAGE, v=0x1000000 + PAGE, k_scales=0x1000000 + 2 * PAGE - 16),
])
def test_kv_write_refuses_a_cache_whose_parts_overlap(S, kw):
    assert _write(S, **kw) == S.ERR_INVALID_ARG and "overlap" in S.F["spear_last_error"]().decode()


@pytest.mark.parametrize("kw", [
    {}, dict(v=0x1000000 + 10 * PAGE), dict(v=0x1000000 - 10 * PAGE), dict(page_stride=2 * PAGE, v=0x1000000 + PAGE),
    dict(page_stride=2 * PAGE, v=0x1000000 - PAGE), dict(page_stride=2 * PAGE, v=0x1000000 + 5 * PAGE),
    dict(page_stride=4 * PAGE, scale_stride=2 * PAGE, v=0x1000000 + PAGE, k_scales=0x1000000 + 2 * PAGE,
         v_scales=0x1000000 + 2 * PAGE + PAGE_SCALES),
])
def test_kv_write_takes_parts_beside_one_another(S, kw):
    assert _write(S, **kw) == S.ERR_UNSUPPORTED_SHAPE, S.F["spear_last_error"]().decode()
