"""Writing tokens into the quantised paged cache and reading them back: codes,
scales and values bit for bit as the oracle's."""
import numpy as np
import pytest
import torch

from oracle import spear_oracle as O
from tests.decoder_cases import KINDS, bf16_tensor, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


def _ws(S):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return ws


def _values(rng, n, heads, dim):
    """Rows of every sort: ordinary, outliers, zeros, tiny, huge, on the grid's ties."""
    x = rng.standard_normal((n, heads, dim)).astype(np.float32)
    for i in range(n):
        sort = i % 8
        if sort == 1:
            x[i] *= np.where(rng.random((heads, dim)) < 0.02, 50.0, 1.0)
        elif sort == 2:
            x[i] = 0.0
        elif sort == 3:
            x[i] *= 1e-9                       # scale 0 in fp16
        elif sort == 4:
            x[i] *= 1e30                       # scale saturates
        elif sort == 5:
            x[i] = (rng.integers(-14, 15, (heads, dim)) / 2.0)
            x[i, :, 0] = 7.0                   # int4: s = 1, halves are ties
        elif sort == 6:
            x[i] *= 1e-6                       # subnormal fp16 scale
        elif sort == 7:
            x[i] *= 10.0 ** rng.uniform(-3, 3, (heads, 1))
    return x


def _read_pages(cache, kind, slots):
    page, off = slots // cache.page_size, slots % cache.page_size
    got = []
    for codes, sc in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        got.append((codes[page, :, off].cpu(), None if kind == "bf16" else sc[page, :, off].cpu()))
    return got


def _expected(x, kind):
    """stored codes, scale, float64 value of x (bf16 tensor)"""
    v = f64(x)
    if kind == "bf16":
        return x.cpu(), None, v
    q, s = O.kv_quantize(v, kind)
    return torch.from_numpy(q if kind == "int8" else O.kv_pack4(q)), torch.from_numpy(s), O.kv_values(q, s)


def _bf16_of(v):
    with np.errstate(over="ignore", invalid="ignore"):
        return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,page,n", [(1, 16, 1), (3, 16, 50), (8, 64, 129), (2, 1024, 1025)])
def test_write_and_read_back(S, kind, dim, heads, page, n):
    rng = np.random.default_rng(dim + n)
    cache = S.make_kv_cache(KINDS[kind], (n + 40) // page + 2, page, heads, dim)
    ws = _ws(S)
    k, v = bf16_tensor(_values(rng, n, heads, dim)), bf16_tensor(_values(rng, n, heads, dim))
    slots = torch.from_numpy(rng.permutation(cache.n_pages * page)[:n].astype(np.int32)).cuda()
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales) if t is not None]
    S.kv_write(cache, k, v, slots, ws)
    k_back, v_back = S.kv_read(cache, slots, ws)
    assert S.read_status(ws) == S.OK
    for x, back, (codes, sc) in zip((k, v), (k_back, v_back), _read_pages(cache, kind, slots.long())):
        want, ws_, val = _expected(x, kind)
        assert torch.equal(codes, want)
        if sc is not None:
            assert torch.equal(sc.view(torch.int16), ws_.view(torch.int16))
        assert torch.equal(back.cpu(), _bf16_of(val))
    # nothing else was touched
    rest = torch.ones(cache.n_pages * page, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    at = rest.nonzero()[:, 0]
    for t, b in zip([t for t in (cache.k, cache.v, cache.k_scales, cache.v_scales) if t is not None], before):
        assert torch.equal(t[at // page, :, at % page], b[at // page, :, at % page])


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_every_maximum_and_its_ties(S, kind):
    # a row for every finite bf16 magnitude as the row's largest; below it values of the
    # next eight octaves, and those next to and on the halves between codes
    rng = np.random.default_rng(6)
    top = np.arange(0x7F80, dtype=np.int64)[:, None]
    bits = np.maximum(top - rng.integers(0, 0x400, (0x7F80, 64)), 0)
    with np.errstate(over="ignore"):
        s = O.kv_quantize(O.bf16_to_f64(top.astype(np.uint16))[:, None], kind)[1].astype(np.float64)
    halves = (rng.integers(0, 127 if kind == "int8" else 7, (0x7F80, 32)) + 0.5) * s.reshape(-1, 1)
    half_bits = O.f32_to_bf16_bits_rne(halves.astype(np.float32)).astype(np.int64) + rng.integers(-1, 2, (0x7F80, 32))
    bits[:, 32:] = np.clip(half_bits, 0, top)
    bits[:, 0] = top[:, 0]
    signed = (bits | rng.integers(0, 2, bits.shape) << 15).astype(np.uint16)
    x = torch.from_numpy(signed.view(np.int16)).view(torch.bfloat16).view(0x7F80, 1, 64).cuda()
    cache = S.make_kv_cache(KINDS[kind], 0x7F80 // 64, 64, 1, 64)
    slots = torch.arange(0x7F80, dtype=torch.int32, device="cuda")
    ws = _ws(S)
    S.kv_write(cache, x, x, slots, ws)
    want, sc, _ = _expected(x, kind)
    for codes, got in _read_pages(cache, kind, slots.long()):
        assert torch.equal(codes, want)
        assert torch.equal(got.view(torch.int16), sc.view(torch.int16))


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_many_ordinary_rows_bit_for_bit(S, kind):
    # enough quotients that some lie next to a tie
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((4096, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
    cache = S.make_kv_cache(KINDS[kind], 64, 64, 4, 128)
    slots = torch.arange(4096, dtype=torch.int32, device="cuda")
    ws = _ws(S)
    S.kv_write(cache, x, x, slots, ws)
    want, sc, _ = _expected(x, kind)
    for codes, s in _read_pages(cache, kind, slots.long()):
        assert torch.equal(codes, want) and torch.equal(s, sc)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_nan_and_infinite_values(S, kind):
    x = np.ones((4, 2, 64), dtype=np.float32)
    x[0, 0, 5], x[1, 1, 7], x[2, 0, 0], x[3, 1, 63] = np.nan, np.inf, -np.inf, np.nan
    x[3, 1, 62] = np.inf
    t = bf16_tensor(x)
    cache = S.make_kv_cache(KINDS[kind], 1, 16, 2, 64)
    ws = _ws(S)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    S.kv_write(cache, t, t, slots, ws)
    back, _ = S.kv_read(cache, slots, ws)
    if kind == "bf16":
        assert torch.equal(back.view(torch.int16), t.view(torch.int16))
        return
    _, _, val = _expected(t, kind)
    want = _bf16_of(val)
    assert torch.equal(torch.isnan(back.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(back.cpu()), torch.nan_to_num(want))
    assert torch.isnan(back[0, 0]).all() and not torch.isnan(back[0, 1]).any()


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_skipped_and_bad_slots(S, kind):
    cache = S.make_kv_cache(KINDS[kind], 3, 16, 2, 64)
    ws = _ws(S)
    x = bf16_tensor(np.random.default_rng(1).standard_normal((5, 2, 64)))
    slots = torch.tensor([4, -1, 47, -(1 << 31), 20], dtype=torch.int32, device="cuda")
    S.kv_write(cache, x, x, slots, ws)
    assert S.read_status(ws) == S.OK
    live = cache.k.reshape(3, 2, 16, -1).ne(0).any(-1).any(1).flatten().nonzero()[:, 0].tolist()
    if kind != "int4":
        assert live == [4, 20, 47]
    before = cache.k.clone(), cache.v.clone()
    for bad in (48, 1 << 30, 2147483647):
        S.kv_write(cache, x[:1], x[:1], torch.tensor([bad], dtype=torch.int32, device="cuda"), ws)
        assert S.read_status(ws) == S.ERR_DEVICE_CHECK
        k, v = S.kv_read(cache, torch.tensor([bad, 20], dtype=torch.int32, device="cuda"), ws)
        assert S.read_status(ws) == S.ERR_DEVICE_CHECK
        assert torch.all(k[0] == 0) and torch.all(v[0] == 0) and torch.any(k[1] != 0)
    assert torch.equal(before[0], cache.k) and torch.equal(before[1], cache.v)
    k, v = S.kv_read(cache, torch.tensor([-1, 4, 4, -5], dtype=torch.int32, device="cuda"), ws)
    assert S.read_status(ws) == S.OK
    assert torch.all(k[0] == 0) and torch.all(v[3] == 0) and torch.equal(k[1], k[2]) and torch.any(k[1] != 0)


def test_column_ranges_of_one_projection(S):
    # q, k and v as one projection's output: k and v are column ranges of it
    H, D, n = 2, 64, 7
    wide = bf16_tensor(np.random.default_rng(2).standard_normal((n, 4 * H * D)))
    k, v = wide[:, 2 * H * D:3 * H * D], wide[:, 3 * H * D:]
    ws = _ws(S)
    slots = torch.arange(n, dtype=torch.int32, device="cuda") + 3
    a, b = S.make_kv_cache(S.KV_INT8, 2, 16, H, D), S.make_kv_cache(S.KV_INT8, 2, 16, H, D)
    S.kv_write(a, k, v, slots, ws)
    S.kv_write(b, k.contiguous().view(n, H, D), v.contiguous().view(n, H, D), slots, ws)
    for s, t in ((a.k, b.k), (a.v, b.v), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
        assert torch.equal(s, t)
    assert S.read_status(ws) == S.OK and torch.any(a.k != 0)


def test_pages_apart_share_one_allocation(S):
    # K and V of a page side by side in one buffer
    n_pages, H, P, D = 4, 2, 16, 64
    both = torch.full((n_pages, 2, H, P, D), 99, dtype=torch.int8, device="cuda")
    sc = torch.full((n_pages, 2, H, P), 9.0, dtype=torch.float16, device="cuda")
    c = S.kv_cache_from_parts(both[:, 0], both[:, 1], sc[:, 0], sc[:, 1])
    d = S.make_kv_cache(S.KV_INT8, n_pages, P, H, D)
    x = bf16_tensor(np.random.default_rng(3).standard_normal((n_pages * P, H, D)))
    slots = torch.arange(n_pages * P, dtype=torch.int32, device="cuda")
    ws = _ws(S)
    for cache in (c, d):
        S.kv_write(cache, x, -x, slots, ws)
    assert torch.equal(c.k, d.k) and torch.equal(c.v, d.v) and torch.equal(c.v_scales, d.v_scales)
    for a, b in zip(S.kv_read(c, slots, ws), S.kv_read(d, slots, ws)):
        assert torch.equal(a, b)


def test_nothing_to_do_graph_and_stream(S):
    cache = S.make_kv_cache(S.KV_INT4, 4, 16, 2, 64)
    ws = _ws(S)
    x = bf16_tensor(np.random.default_rng(4).standard_normal((6, 2, 64)))
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    S.kv_write(cache, x[:0], x[:0], slots[:0], ws)
    assert S.kv_read(cache, slots[:0], ws)[0].shape == (0, 2, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    S.kv_write(cache, x, x, slots, ws, stream=st)
    k, v = S.kv_read(cache, slots, ws, stream=st)
    st.synchronize()
    want = _bf16_of(_expected(x, "int4")[2])
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    # captured: replays take the values and slots that the buffers then hold
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            S.kv_write(cache, x, x, slots, ws)
            S.kv_read(cache, slots, ws, k_out=ko, v_out=vo)
    x.mul_(3.0)
    slots.add_(11)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ko.cpu(), _bf16_of(_expected(x, "int4")[2])) and torch.equal(ko, vo)


def test_offsets_past_32_bits(S):
    n_pages, page, heads, dim = 5 << 13, 64, 8, 256
    k = torch.empty((n_pages, heads, page, dim), dtype=torch.int8, device="cuda")
    sc = torch.empty((n_pages, heads, page), dtype=torch.float16, device="cuda")
    assert k.numel() > 1 << 32
    cache = S.kv_cache_from_parts(k, torch.empty_like(k), sc, torch.empty_like(sc))
    x = bf16_tensor(np.random.default_rng(5).standard_normal((3, heads, dim)))
    slots = torch.tensor([n_pages * page - 1, n_pages * page - 64, 5], dtype=torch.int32, device="cuda")
    ws = _ws(S)
    S.kv_write(cache, x, x, slots, ws)
    back, _ = S.kv_read(cache, slots, ws)
    assert S.read_status(ws) == S.OK
    assert torch.equal(back.cpu(), _bf16_of(_expected(x, "int8")[2]))


def test_binding_refusals(S):
    cache = S.make_kv_cache(S.KV_INT8, 2, 16, 2, 64)
    ws = _ws(S)
    x, slots = bf16_tensor(np.zeros((3, 2, 64))), torch.arange(3, dtype=torch.int32, device="cuda")
    for args in ((x.float(), x, slots, ws), (x, x[:2], slots, ws), (x, x, slots.long(), ws), (x, x, slots[:2], ws),
                 (x.view(3, 128)[:, :64], x, slots, ws), (x.cpu(), x, slots, ws), (x, x, slots, ws.cpu())):
        with pytest.raises((TypeError, ValueError)):
            S.kv_write(cache, *args)
    with pytest.raises(S.SpearError):
        S.kv_write(cache, x, x, slots, ws[:64])
    with pytest.raises(S.SpearError):
        S.kv_write(cache, x[:1].expand(3, 2, 64), x, slots, ws)       # rows on top of one another
    with pytest.raises(ValueError):
        S.kv_read(cache, slots, ws, k_out=x.float())
    p = torch.zeros((4, 2, 16, 64), dtype=torch.int8, device="cuda")
    s = torch.zeros((4, 2, 16), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        S.kv_cache_from_parts(p.transpose(1, 2).contiguous().transpose(1, 2), p, s, s)
    with pytest.raises(ValueError):
        S.kv_cache_from_parts(p, p.clone(), s.float(), s)
    with pytest.raises(ValueError):
        S.kv_cache_from_parts(p[:1].expand(4, 2, 16, 64), p[:1].expand(4, 2, 16, 64), s, s)
    with pytest.raises(S.SpearError):
        S.kv_cache_from_parts(p[..., :32].contiguous(), p[..., :32].contiguous(), s, s)
