"""Caches that are dropped while another stream still works on them, and caches
whose parts share an allocation."""
import numpy as np
import pytest
import torch

from tests.decoder_cases import Filled, bf16_tensor

pytestmark = pytest.mark.gpu

DELAY = 40_000_000     # cycles that a side stream waits before it works: some 20 ms


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


def _fill_like(tensors):
    """New tensors of these sizes on the current stream, written over at once."""
    made = [torch.empty(t[0], dtype=t[1], device="cuda") for t in tensors]
    for t in made:
        t.view(torch.uint8).fill_(0x5A)
    return made


def _shapes(cache):
    return [(t.shape, t.dtype) for t in (cache.k, cache.v, cache.k_scales, cache.v_scales) if t is not None]


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_attention_on_a_stream_outlives_the_cache(S, kind):
    f = Filled(S, kind, [3000, 700], 2, 128, 16, seed=1)
    q = bf16_tensor(np.random.default_rng(2).standard_normal((2, 8, 128)))
    ws = S.make_attn_workspace(f.cache, 8)
    want = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)
    shapes, side = _shapes(f.cache), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    got = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, stream=side)
    f.cache = None
    made = _fill_like(shapes)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(torch.all(t.view(torch.uint8) == 0x5A) for t in made)


@pytest.mark.parametrize("kind", ["BF16", "INT8", "INT4"])
def test_a_write_on_a_stream_reaches_no_later_tensor(S, kind):
    cache = S.make_kv_cache(getattr(S, "KV_" + kind), 64, 16, 4, 128)
    ws = S.make_attn_workspace(cache, 4)
    n = 1024
    k, v = (bf16_tensor(np.random.default_rng(i).standard_normal((n, 4, 128))) for i in (3, 4))
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    S.kv_write(cache, k, v, slots, ws)
    want = S.kv_read(cache, slots, ws)
    shapes, side = _shapes(cache), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    S.kv_write(cache, k, v, slots, ws, stream=side)
    got = S.kv_read(cache, slots, ws, stream=side)
    del cache
    made = _fill_like(shapes)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.all(t.view(torch.uint8) == 0x5A) for t in made)


# ---- caches whose parts share an allocation ---------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_keys_and_values_of_a_page_side_by_side(S, kind):
    f = Filled(S, kind, [200, 33], 2, 64, 16, seed=5)
    c = f.cache
    pages = torch.stack([c.k, c.v], dim=1)                    # n_pages x 2 x heads x page x dim
    scales = None if kind == "bf16" else torch.stack([c.k_scales, c.v_scales], dim=1)
    f.cache = S.kv_cache_from_parts(pages[:, 0], pages[:, 1], *(() if scales is None else (scales[:, 0], scales[:, 1])))
    ws = S.make_attn_workspace(f.cache, 4)
    q = bf16_tensor(np.random.default_rng(6).standard_normal((2, 4, 64)))
    f.check(S, q, S.attn_decode(q, f.cache, f.table, f.seq_lens, ws), None, 0.125, ws)
    k, v = (bf16_tensor(np.random.default_rng(i).standard_normal((40, 2, 64))) for i in (7, 8))
    slots = (f.table[0, :3].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:40].to(torch.int32)
    S.kv_write(f.cache, k, v, slots, ws)
    got = S.kv_read(f.cache, slots, ws)
    S.kv_write(c, k, v, slots, ws)                            # the same into pages apart
    assert all(torch.equal(a, b) for a, b in zip(got, S.kv_read(c, slots, ws)))
    bits = [t.contiguous().view(torch.uint8) for t in (pages[:, 0], c.k, pages[:, 1], c.v)]   # free places hold NaN
    assert torch.equal(bits[0], bits[1]) and torch.equal(bits[2], bits[3]) and S.read_status(ws) == S.OK


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_one_array_for_keys_and_values_is_read_and_not_written(S, kind):
    f = Filled(S, kind, [90, 20], 2, 64, 16, seed=9)
    c = f.cache
    f.cache = S.kv_cache_from_parts(c.k, c.k, c.k_scales, c.k_scales)
    f.v = f.k
    ws = S.make_attn_workspace(f.cache, 4)
    q = bf16_tensor(np.random.default_rng(10).standard_normal((2, 4, 64)))
    f.check(S, q, S.attn_decode(q, f.cache, f.table, f.seq_lens, ws), None, 0.125, ws)
    k = bf16_tensor(np.random.default_rng(11).standard_normal((2, 2, 64)))
    with pytest.raises(S.SpearError):
        S.kv_write(f.cache, k, k, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), ws)


def test_calls_on_a_given_stream_are_captured(S):
    f = Filled(S, "int8", [700, 33], 2, 64, 16, seed=12)
    ws = S.make_attn_workspace(f.cache, 4)
    q = bf16_tensor(np.random.default_rng(13).standard_normal((2, 4, 64)))
    want = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)
    out, side, graph = torch.zeros_like(want), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, out=out, stream=side)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
