"""Caches that are dropped while another stream still works on them."""
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
