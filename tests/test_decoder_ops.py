"""Key-value cache, attention and block norms without a GPU: the oracle's pins,
size queries, argument validation before any launch, the struct's layout."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import spear_oracle as O
from tests.conftest import ROOT


@pytest.fixture(scope="module")
def S():
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


# ---- oracle pins --------------------------------------------------------------
def test_kv_quantize_by_hand():
    # max 7 -> s = 1; 0.5 and 1.5 are ties (to even); -3.4 -> -3
    q, s = O.kv_quantize([[7.0, 0.5, 1.5, -3.4]], "int4")
    assert s[0] == 1.0 and q[0].tolist() == [7, 0, 2, -3]
    q, s = O.kv_quantize([[254.0, -254.0, 1.0, 3.0]], "int8")       # s = 2
    assert s[0] == 2.0 and q[0].tolist() == [127, -127, 0, 2]
    q, s = O.kv_quantize([[0.0, -0.0]], "int8")
    assert s[0] == 1.0 and q[0].tolist() == [0, 0]
    q, s = O.kv_quantize([[1.0, np.nan]], "int8")
    assert np.isnan(s[0]) and q[0].tolist() == [0, 0]
    q, s = O.kv_quantize([[np.inf, 1.0, -np.inf]], "int4")
    assert s[0] == 65504.0 and q[0].tolist() == [7, 0, -7]
    assert O.kv_pack4(np.array([[-7, 7, 0, 1]], dtype=np.int8)).tolist() == [[0xF1, 0x98]]


def test_kv_quantize_error_is_half_a_step():
    x = np.random.default_rng(0).standard_normal((50, 64)).astype(np.float32)
    for kind in ("int8", "int4"):
        q, s = O.kv_quantize(x, kind)
        # the fp16 scale may be 2^-11 short of max / Q, which the clamp then costs the largest value
        assert np.all(np.abs(O.kv_values(q, s) - x) <= s.astype(np.float64)[:, None] * (0.5 + 127 * 2.0 ** -11) + 1e-12)


def test_attend_closed_forms():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, lse, p = O.attend(0 * q, k, v, 1.0)                        # equal scores: the mean
    assert np.allclose(out[3], v[:, 1].mean(0)) and np.allclose(lse, np.log(5))
    out, lse, _ = O.attend(q, k[:1], v[:1], 0.5)                    # one token: its value
    assert np.allclose(out[1], v[0, 0]) and np.isclose(lse[2], 0.5 * q[2] @ k[0, 1])
    out, lse, _ = O.attend(q, k[:0], v[:0], 1.0)                    # none
    assert np.all(out == 0) and np.all(lse == -np.inf)
    brute = sum(np.exp(q[2] @ k[t, 1]) * v[t, 1] for t in range(5)) / sum(np.exp(q[2] @ k[t, 1]) for t in range(5))
    assert np.allclose(O.attend(q, k, v, 1.0)[0][2], brute)


def test_block_norm_oracle():
    x, y = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    xo, h = O.block_norm(x, None, None, None, 1.0, 1.0, None, 0.0)
    assert np.allclose(h, x / np.sqrt(12.5)) and np.allclose(xo, x)
    xo, h = O.block_norm(x, 5 * y, np.array([2.0, 3.0]), np.array([0.5, 1.0]), 2.0, 10.0, np.array([1.0, 2.0]), 0.0)
    assert np.allclose(xo, [[6 + 10, 8 - 30]])
    assert np.allclose(h, xo / np.sqrt((16 ** 2 + 22 ** 2) / 2) * [1.0, 2.0])


# ---- size queries, layout -----------------------------------------------------------
def test_page_sizes(S):
    B, C = S.F["spear_kv_page_bytes"], S.F["spear_kv_page_scales"]
    assert B(S.KV_BF16, 16, 8, 128) == 16 * 8 * 256 and C(S.KV_BF16, 16, 8, 128) == 0
    assert B(S.KV_INT8, 32, 8, 128) == 32 * 8 * 128 and C(S.KV_INT8, 32, 8, 128) == 256
    assert B(S.KV_INT4, 1024, 1, 64) == 1024 * 32 and C(S.KV_INT4, 1024, 1, 64) == 1024
    for bad in ((3, 16, 8, 128), (-1, 16, 8, 128), (0, 8, 8, 128), (0, 24, 8, 128), (0, 2048, 8, 128), (0, 16, 0, 128),
                (0, 16, 1025, 128), (0, 16, 8, 96)):
        assert B(*bad) == 0 and C(*bad) == 0


def test_cache_struct_matches_the_header(S, tmp_path):
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    fields = [n for n, _ in S.KVCacheStruct._fields_]
    lines = ['#include <stdio.h>', '#include "spear.h"', "int main(void) {",
             '  printf("%zu %d %d %d\\n", sizeof(spear_kv_cache), SPEAR_KV_BF16, SPEAR_KV_INT8, SPEAR_KV_INT4);']
    lines += [f'  printf("%zu\\n", offsetof(spear_kv_cache, {f}));' for f in fields] + ["  return 0;", "}"]
    src, exe = tmp_path / "kv.c", tmp_path / "kv"
    src.write_text("\n".join(lines))
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(t) for t in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got[:4] == [ctypes.sizeof(S.KVCacheStruct), S.KV_BF16, S.KV_INT8, S.KV_INT4]
    assert got[4:] == [getattr(S.KVCacheStruct, f).offset for f in fields]


# ---- refusals at the C ABI (nothing is launched) -------------------------------------
def _cache(S, **kw):
    d = dict(kind=1, n_pages=10, page_size=16, n_heads=8, head_dim=128, k=0x10000, v=0x20000, k_scales=0x30000,
             v_scales=0x40000, page_stride=0, scale_stride=0)
    d.update(kw)
    return S.KVCacheStruct(**d)


BAD_CACHES = [
    (dict(kind=3), 2), (dict(kind=-1), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(n_heads=0), 2),
    (dict(head_dim=80), 2), (dict(n_pages=0), 2), (dict(n_pages=1 << 27, page_size=16), 2), (dict(k=None), 1),
    (dict(v=None), 1), (dict(k_scales=None), 1), (dict(v_scales=None), 1), (dict(k=0x10008), 3),
    (dict(v_scales=0x40002), 3), (dict(page_stride=16), 1), (dict(page_stride=16 * 8 * 128 + 8), 1),
    (dict(page_stride=-16), 1), (dict(scale_stride=120), 1), (dict(scale_stride=129), 1),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(S, kw, code):
    c = ctypes.byref(_cache(S, **kw))
    assert S.F["spear_kv_write"](c, 0x1000, 1024, 0x2000, 1024, 0x3000, 4, 0x4000, 256, None) == code
    assert S.F["spear_last_error"]().decode()
    assert S.F["spear_kv_read"](c, 0x3000, 4, 0x1000, 0x2000, 0x4000, 256, None) == code
    assert S.F["spear_attn_decode"](c, 0x1000, 4096, 2, 32, 0x2000, 4, 4, 0x3000, 0.1, 0x5000, 4096, None, 0x6000,
                                    1 << 30, None) == code
    assert S.F["spear_attn_workspace_bytes"](c, 32) == 0


def test_cache_without_scales_is_fine_for_bf16(S):
    assert S.F["spear_attn_workspace_bytes"](ctypes.byref(_cache(S, kind=0, k_scales=None, v_scales=None)), 8) >= 256
    assert S.F["spear_attn_workspace_bytes"](ctypes.byref(_cache(S, page_stride=1 << 20, scale_stride=1 << 10)), 8) >= 256


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(ws=None), 1),
    (dict(k=0x1008), 3), (dict(slots=0x3002), 3), (dict(ws=0x4004), 3), (dict(ld_k=1016), 1), (dict(ld_v=1028), 1),
    (dict(ws_bytes=255), 4), (dict(n=0, k=None), 0),
])
def test_kv_write_refusals(S, kw, code):
    d = dict(k=0x1000, ld_k=1024, v=0x2000, ld_v=1024, slots=0x3000, n=4, ws=0x4000, ws_bytes=256)
    d.update(kw)
    rc = S.F["spear_kv_write"](ctypes.byref(_cache(S)), d["k"], d["ld_k"], d["v"], d["ld_v"], d["slots"], d["n"],
                               d["ws"], d["ws_bytes"], None)
    assert rc == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(slots=None), 1), (dict(k=None), 1), (dict(v=0x2002), 3), (dict(ws_bytes=0), 4),
    (dict(n=0, slots=None), 0),
])
def test_kv_read_refusals(S, kw, code):
    d = dict(slots=0x3000, n=4, k=0x1000, v=0x2000, ws=0x4000, ws_bytes=256)
    d.update(kw)
    assert S.F["spear_kv_read"](ctypes.byref(_cache(S)), d["slots"], d["n"], d["k"], d["v"], d["ws"], d["ws_bytes"],
                                None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), 2), (dict(heads=12), 2), (dict(heads=1032), 2), (dict(seqs=-1), 2), (dict(seqs=4097), 2),
    (dict(seqs=0, q=None), 0), (dict(q=None), 1), (dict(out=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(ws=None), 1), (dict(q=0x1008), 3), (dict(out=0x5008), 3), (dict(table=0x2002), 3), (dict(lse=0x7002), 3),
    (dict(ws=0x6008), 3), (dict(ld_q=4088), 1), (dict(ld_q=4100), 1), (dict(ld_out=0), 1), (dict(max_pages=0), 1),
    (dict(ld_table=3), 1), (dict(max_pages=1 << 27, ld_table=1 << 27), 2), (dict(ws_bytes=255), 4),
    (dict(out=0x1000), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
])
def test_attn_refusals(S, kw, code):
    d = dict(q=0x1000, ld_q=4096, seqs=2, heads=32, table=0x2000, max_pages=4, ld_table=4, lens=0x3000, scale=0.1,
             out=0x500000, ld_out=4096, lse=None, ws=0x600000, ws_bytes=1 << 30)
    d.update(kw)
    if kw.get("out") == 0x5008:
        d["out"] = 0x500008
    rc = S.F["spear_attn_decode"](ctypes.byref(_cache(S)), d["q"], d["ld_q"], d["seqs"], d["heads"], d["table"],
                                  d["max_pages"], d["ld_table"], d["lens"], d["scale"], d["out"], d["ld_out"],
                                  d["lse"], d["ws"], d["ws_bytes"], None)
    assert rc == code, S.F["spear_last_error"]().decode()


@pytest.mark.parametrize("kw,code", [
    (dict(K=12), 2), (dict(K=0), 2), (dict(K=16392), 2), (dict(M=-1), 2), (dict(M=(1 << 20) + 1), 2),
    (dict(M=0, x=None), 0), (dict(x=None), 1), (dict(xo=None, h=None), 1), (dict(y=None), 1),
    (dict(y=None, xo=None, post=None), 1), (dict(gate_ld=56), 1), (dict(gate_ld=68), 1), (dict(gate_ld=-64), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=0x10008), 3), (dict(pre=0x5008), 3),
    (dict(h=0x30000), 1),             # h is x_out
    (dict(xo=0x10010), 1),            # shifted against x
    (dict(h=0x20100), 1),             # shifted against y
    (dict(xo=0x6000), 1),             # the gate's rows
    (dict(h=0x5000), 1),              # a weight
])
def test_block_norm_refusals(S, kw, code):
    d = dict(x=0x10000, y=0x20000, M=4, K=64, post=0x4000, gate=0x6000, gate_ld=64, a=1.0, b=1.0, pre=0x5000, eps=1e-6,
             xo=0x30000, h=0x38000)
    d.update(kw)
    rc = S.F["spear_block_norm"](d["x"], d["y"], d["M"], d["K"], d["post"], d["gate"], d["gate_ld"], d["a"], d["b"],
                                 d["pre"], d["eps"], d["xo"], d["h"], None)
    assert rc == code, S.F["spear_last_error"]().decode()


# ---- refusals of the binding ----------------------------------------------------------
@pytest.mark.parametrize("out,ld,seqs", [
    (0x1000, 4096, 1), (0x1010, 4096, 2), (0x2FF0, 4096, 1), (0x1000 + 4096, 6144, 2), (0x1000 + 8192, 4104, 2),
    (0x1000 + 8192 - 16, 16384, 3), (0x1000 + 2 * 16384 - 8192 + 16, 16384, 3),
])
def test_attn_refuses_overlaps_of_q_and_out(S, out, ld, seqs):
    rc = S.F["spear_attn_decode"](ctypes.byref(_cache(S)), 0x1000, ld, seqs, 32, 0x900000, 4, 4, 0xA00000, 0.1, out, ld,
                                  None, 0x600000, 255, None)
    assert rc == 1 and "overlap" in S.F["spear_last_error"]().decode()


@pytest.mark.parametrize("out,ld,seqs", [
    (0x1000 + 8192, 4096, 1), (0x1000 + 8192, 8192, 5), (0x1000 + 2 * 16384 - 8192, 16384, 3),
    (0x1000 + 32768 + 8192, 16384, 3), (0x100000 - 8192, 4096, 1),
])
def test_attn_takes_q_and_out_as_columns_of_the_same_rows(S, out, ld, seqs):
    # past the check, the workspace is refused
    assert S.F["spear_attn_decode"](ctypes.byref(_cache(S)), 0x1000, ld, seqs, 32, 0x900000, 4, 4, 0xA00000, 0.1, out, ld,
                                    None, 0x600000, 255, None) == 4


@pytest.mark.parametrize("v", [0x1000, 0x1010, 0x1000 + 4 * 1024 * 2 - 16, 0x1000 - 16])
def test_kv_read_refuses_overlapping_outputs(S, v):
    assert S.F["spear_kv_read"](ctypes.byref(_cache(S)), 0x300000, 4, 0x1000, v, 0x400000, 256, None) == 1


def test_binding_refuses_host_tensors_and_wrong_types(S):
    z = torch.zeros
    with pytest.raises(TypeError):
        S.kv_cache_from_parts(z((2, 4, 16, 64)), z((2, 4, 16, 64)))
    with pytest.raises(ValueError):
        S.kv_cache_from_parts(z((2, 4, 16, 64), dtype=torch.bfloat16), z((2, 4, 16, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        S.kv_cache_from_parts(z((2, 4, 16, 64), dtype=torch.int8), z((2, 4, 16, 64), dtype=torch.int8))
    with pytest.raises(ValueError):
        S.kv_cache_from_parts(z((2, 16, 64), dtype=torch.bfloat16), z((2, 16, 64), dtype=torch.bfloat16))
    with pytest.raises(S.SpearError):
        S.make_kv_cache(S.KV_INT8, 4, 20, 8, 128)
    with pytest.raises(S.SpearError):
        S.make_kv_cache(S.KV_INT8, 0, 16, 8, 128)
    with pytest.raises(ValueError):
        S.block_norm(z((2, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        S.block_norm(z((2, 64)))


def test_advance_gives_slots_up_to_the_last_page(S):
    from types import SimpleNamespace

    from w4_gemm_gated_b200 import decoder
    table = torch.tensor([[5, 2], [0, 7], [3, 1], [4, 6]], dtype=torch.int32)
    state = decoder.StepState([SimpleNamespace(page_size=16)], table, torch.tensor([0, 16, 31, 32], dtype=torch.int32),
                              torch.zeros(4, dtype=torch.int32), None, None)
    decoder.advance(state)
    assert state.slots.tolist() == [80, 112, 31, -1] and state.seq_lens.tolist() == [1, 17, 32, 33]
    decoder.advance(state)
    assert state.slots.tolist() == [81, 113, -1, -1] and state.seq_lens.tolist() == [2, 18, 33, 34]
    assert state.slots.dtype == torch.int32


def test_a_cache_keeps_its_tensors(S):
    # its struct holds their addresses
    k, v = (torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16) for _ in range(2))
    cache = S.KVCache(S.KV_BF16, 2, 16, 1, 64, k, v)
    with pytest.raises(AttributeError):
        cache.k = torch.zeros_like(k)
    assert cache.k is k and cache.struct.k == k.data_ptr() and cache.struct.page_stride == 16 * 64 * 2
