"""Norms around a block with its gate and residual scale, against float64."""
import numpy as np
import pytest
import torch

from oracle import spear_oracle as O
from tests.decoder_cases import HALF, bf16_tensor, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


def _inputs(M, K, post, gate, pre, seed, scale=1.0):
    r = np.random.default_rng(seed)
    t = {"x": bf16_tensor(r.standard_normal((M, K)) * 2 * scale), "y": bf16_tensor(r.standard_normal((M, K)) * scale)}
    t["post_weight"] = bf16_tensor(1 + 0.2 * r.standard_normal(K)) if post else None
    t["pre_weight"] = bf16_tensor(1 + 0.2 * r.standard_normal(K)) if pre else None
    t["gate"] = {"none": None, "channel": bf16_tensor(r.random(K)), "row": bf16_tensor(r.random((1, K))),
                 "token": bf16_tensor(r.standard_normal((M, K)))}[gate]
    return t


def _check(t, xo, h, a, b, eps, x=None, y=None):
    x64, y64 = f64(t["x"] if x is None else x), f64(t["y"] if y is None else y)
    post, gate, pre = (None if t[n] is None else f64(t[n]) for n in ("post_weight", "gate", "pre_weight"))
    want_x, want_h = O.block_norm(x64, y64, post, gate, a, b, pre, eps)
    # fp32: the mean of squares to (K / 256 + 20) 2^-24 in a chain of partial sums,
    # a few roundings more; x_out's error is relative to its terms, which may cancel
    K = x64.shape[1]
    rel = (K / 256 + 64) * 2.0 ** -24
    terms = np.abs(a * x64) + np.abs(want_x - a * x64)
    tol_x = HALF * np.abs(want_x) + rel * terms + 1e-37
    if xo is not None:
        assert np.all(np.abs(f64(xo) - want_x) <= tol_x)
    if h is not None:
        r = 1 / np.sqrt(np.mean(want_x ** 2, -1, keepdims=True) + eps)
        w = 1.0 if pre is None else np.abs(pre)
        # the row's own error enters its root mean square, at most by the same share
        share = rel * np.sqrt(np.mean(terms ** 2, -1, keepdims=True)) * r
        tol_h = HALF * np.abs(want_h) + rel * terms * r * w + (rel + share) * np.abs(want_h) * 2 + 1e-37
        assert np.all(np.abs(f64(h) - want_h) <= tol_h)


@pytest.mark.parametrize("M,K", [(1, 8), (3, 16), (1, 4096), (5, 248), (7, 2056), (2, 8200), (2, 16384), (300, 512),
                                 (33, 1000), (1, 264)])
@pytest.mark.parametrize("post,gate,pre", [(False, "none", True), (True, "channel", True), (True, "token", False),
                                           (False, "row", False)])
def test_sizes_and_options(S, M, K, post, gate, pre):
    t = _inputs(M, K, post, gate, pre, M + K)
    x0, y0 = t["x"].clone(), t["y"].clone()
    xo, h = S.block_norm(**t, residual_scale=0.7, block_scale=-1.3, eps=1e-5)
    _check(t, xo, h, np.float32(0.7), np.float32(-1.3), 1e-5)
    assert torch.equal(t["x"], x0) and torch.equal(t["y"], y0)


@pytest.mark.parametrize("K", [64, 4096])
def test_norm_alone(S, K):
    t = _inputs(9, K, False, "none", True, K)
    same, h = S.block_norm(t["x"], pre_weight=t["pre_weight"], eps=1e-6)
    assert same is t["x"]
    _check({**t, "y": torch.zeros_like(t["x"])}, None, h, 1.0, 0.0, 1e-6)


def test_update_alone_and_in_place(S):
    for K in (136, 4096):
        t = _inputs(11, K, True, "token", True, K)
        xo, none = S.block_norm(**t, norm=False)
        assert none is None
        _check(t, xo, None, 1.0, 1.0, 1e-6)
        want, want_h = S.block_norm(**t)
        assert torch.equal(want, xo)
        for names in (("x", "y"), ("y", "x")):
            u = {k: None if v is None else v.clone() for k, v in t.items()}
            got, h = S.block_norm(**u, x_out=u[names[0]], h=u[names[1]])
            assert got is u[names[0]] and torch.equal(got, want) and torch.equal(h, want_h)
        u = t["x"].clone()
        _, h = S.block_norm(u, h=u)
        assert torch.equal(u, S.block_norm(t["x"])[1])


def test_rows_of_zeros_and_extremes(S):
    K = 512
    t = _inputs(6, K, True, "none", True, 5)
    t["x"][0] = 0
    t["y"][0] = 0                            # nothing at all: zeros, not NaN
    t["y"][1] = 0
    t["x"][2] *= 2.0 ** 40
    t["y"][3] *= 2.0 ** -40                  # under eps
    t["x"][4] = 0
    xo, h = S.block_norm(**t, eps=1e-6)
    _check(t, xo, h, 1.0, 1.0, 1e-6)
    assert torch.all(xo[0] == 0) and torch.all(h[0] == 0)


def test_nan_stays_in_its_row(S):
    t = _inputs(4, 256, True, "channel", True, 6)
    t["y"][1, 7] = float("nan")
    t["x"][2, 9] = float("inf")
    xo, h = S.block_norm(**t)
    assert torch.isnan(xo[1]).all() and torch.isnan(h[1]).all()
    assert torch.isinf(xo[2, 9]) and torch.isfinite(xo[2]).sum() == 255
    keep = [0, 3]
    _check({**t, "x": t["x"][keep], "y": t["y"][keep]}, xo[keep], h[keep], 1.0, 1.0, 1e-6)


def test_strided_and_broadcast_gates(S):
    M, K = 10, 264
    t = _inputs(M, K, True, "token", True, 7)
    wide = torch.full((M, 3 * K), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, K:2 * K] = t["gate"]
    want = S.block_norm(**t)
    got = S.block_norm(**{**t, "gate": wide[:, K:2 * K]})
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    one = t["gate"][:1]
    want = S.block_norm(**{**t, "gate": one.repeat(M, 1)})
    for g in (one, one[0], one.expand(M, K)):
        got = S.block_norm(**{**t, "gate": g})
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_stream_and_nothing(S):
    t = _inputs(40, 4096, True, "channel", True, 8)
    want = S.block_norm(**t)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = S.block_norm(**t, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    xo, h = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            S.block_norm(**t, x_out=xo, h=h)
    t["x"].mul_(0.5)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want = S.block_norm(**t)
    assert torch.equal(xo, want[0]) and torch.equal(h, want[1])
    empty = S.block_norm(**{**_inputs(2, 64, True, "channel", True, 9), "x": t["x"][:0, :64].contiguous(),
                            "y": t["y"][:0, :64].contiguous()})
    assert empty[0].shape == (0, 64) and empty[1].shape == (0, 64)


def test_binding_refusals(S):
    t = _inputs(4, 64, True, "token", True, 10)
    for name, bad in (("x", t["x"].float()), ("y", t["y"][:, :32]), ("post_weight", t["post_weight"][:32]),
                      ("pre_weight", t["pre_weight"].float()), ("gate", t["gate"][:2]), ("gate", t["gate"].t()),
                      ("y", t["y"].cpu()), ("x", t["x"][0])):
        with pytest.raises(ValueError):
            S.block_norm(**{**t, name: bad})
    with pytest.raises(S.SpearError):
        S.block_norm(t["x"], post_weight=t["post_weight"])           # nothing to normalise after
    with pytest.raises(S.SpearError):
        S.block_norm(**t, eps=-1.0)
    odd = torch.zeros((4, 12), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(S.SpearError):
        S.block_norm(odd, odd)
