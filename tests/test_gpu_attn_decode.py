"""Attention of one new token per sequence over the paged cache, against the
64-bit oracle: every cache kind, head width and page size, head groups from one
to many, lengths from none to several pages, ragged batches, strides, poisoned
neighbours, bad pages and lengths, graphs, streams, determinism."""
import numpy as np
import pytest
import torch

from tests.decoder_cases import Filled, bf16_tensor, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


def _q(n, heads, dim, seed, scale=1.0):
    return bf16_tensor(np.random.default_rng(seed + 99).standard_normal((n, heads, dim)) * scale)


def _run(S, f, group, seed, scale=None, q_scale=1.0, ws=None):
    H = f.heads * group
    q = _q(len(f.lens), H, f.dim, seed, q_scale)
    ws = S.make_attn_workspace(f.cache, H) if ws is None else ws
    lse = torch.full((len(f.lens), H), 7.0, device="cuda")
    out = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, scale=scale, lse=lse)
    f.check(S, q, out, lse, f.dim ** -0.5 if scale is None else scale, ws)
    return q, out, lse, ws


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 13])
def test_kinds_widths_groups(S, kind, dim, group):
    f = Filled(S, kind, [1, 0, 17, 130, 333], 2, dim, 16, seed=dim + group)
    _run(S, f, group, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
def test_pages_that_end_anywhere(S, kind, page):
    lens = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257]
    f = Filled(S, kind, lens, 1, 64, page, seed=page)
    _run(S, f, 2, seed=2)


@pytest.mark.parametrize("group", [16, 17, 32, 40])
def test_groups_past_one_tile(S, group):
    f = Filled(S, "int8", [5, 70], 1, 128, 16, seed=group)
    _run(S, f, group, seed=3)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [9, 16, 29])
def test_wide_groups_over_many_tokens(S, kind, dim, group):
    # tables that have room for as many tokens as bring pairs of products: short
    # sequences, none, and one over many CTAs
    f = Filled(S, kind, [6000, 0, 1, 130], 1, dim, 64, seed=dim + group, max_pages=1500)
    _run(S, f, group, seed=5)


@pytest.mark.parametrize("kind,lens,heads", [
    ("bf16", [5000], 1), ("int8", [3001, 2], 2), ("int4", [2500], 3),      # one long unit over many workers
    ("int8", [40] * 100, 8),                                               # many short ones
    ("bf16", [9] * 300 + [0] * 20 + [700], 1),                             # many, some empty, one long
])
def test_splits(S, kind, lens, heads):
    f = Filled(S, kind, lens, heads, 64, 16, seed=len(lens))
    _run(S, f, 2, seed=4)


@pytest.mark.parametrize("kind,seqs,tokens", [("int8", 18, 6400), ("bf16", 9, 9600), ("int4", 18, 12800)])
def test_long_units_that_meet_in_a_cta(S, kind, seqs, tokens):
    # units over 17 or 33 CTAs, whose last is the next one's first: each joins its
    # parts in groups of 16, the last group of the one and the first of the other there
    f = Filled(S, kind, [tokens] * seqs, 1, 64 if kind == "bf16" else 128, 64, seed=seqs)
    _, out, lse, ws = _run(S, f, 4, seed=6)
    _, again, lse2, _ = _run(S, f, 4, seed=6, ws=ws)  # the counters are back at zero
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_more_sequences_than_threads(S):
    lens = [(i * 7) % 23 for i in range(1500)]
    f = Filled(S, "int8", lens, 1, 64, 16, seed=3)
    _run(S, f, 1, seed=5)


def test_all_empty(S):
    f = Filled(S, "bf16", [0, 0, 0], 2, 128, 16, seed=3)
    _run(S, f, 4, seed=6)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_sharp_softmax_and_large_scores(S, kind):
    # scores of a hundred and more: one token takes nearly all the weight
    f = Filled(S, kind, [400, 33], 2, 128, 32, seed=8, spread=3.0)
    _run(S, f, 4, seed=7, q_scale=4.0)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("power", [-100, -20, 20, 100])
def test_powers_of_two_between_q_and_scale_change_nothing(S, kind, power):
    f = Filled(S, kind, [5, 130, 700], 2, 128, 16, seed=4)
    q = _q(3, 8, 128, 4)
    ws = S.make_attn_workspace(f.cache, 8)
    want = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, scale=0.1)
    got = S.attn_decode(q * 2.0 ** power, f.cache, f.table, f.seq_lens, ws, scale=0.1 * 2.0 ** -power)
    assert torch.isfinite(want).all() and torch.equal(got, want)


def test_negative_and_zero_scale(S):
    f = Filled(S, "int4", [90], 2, 64, 16, seed=9)
    _run(S, f, 2, seed=8, scale=-0.2)
    _run(S, f, 2, seed=8, scale=0.0)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_pages_inside_a_wider_allocation(S, kind):
    f = Filled(S, kind, [100, 37, 5], 3, 64, 16, seed=10, apart=True)
    assert f.cache.struct.page_stride > 0
    _run(S, f, 2, seed=9)


def test_strided_q_out_and_table(S):
    f = Filled(S, "int8", [50, 20, 75], 2, 64, 16, seed=11)
    H, D = 4, 64
    wide = torch.full((3, 3 * H * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, H * D:2 * H * D] = _q(3, H, D, 3).view(3, -1)
    q = wide[:, H * D:2 * H * D]
    dst = torch.full((3, H * D + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    tab = torch.full((3, f.width + 5), -7, dtype=torch.int32, device="cuda")
    tab[:, 2:2 + f.width] = f.table
    ws = S.make_attn_workspace(f.cache, H)
    out = S.attn_decode(q, f.cache, tab[:, 2:2 + f.width], f.seq_lens, ws, out=dst[:, :H * D])
    f.check(S, q, out, None, 0.125, ws)
    assert torch.all(dst[:, H * D:] == 5.0)


def test_rows_behind_the_last_sequence_stay(S):
    f = Filled(S, "bf16", [20, 40], 2, 64, 16, seed=12)
    q = _q(6, 4, 64, 4)
    out = torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 4), 3.0, device="cuda")
    ws = S.make_attn_workspace(f.cache, 4)
    S.attn_decode(q[:2], f.cache, f.table, f.seq_lens, ws, out=out[:2], lse=lse[:2])
    f.check(S, q[:2], out[:2], lse[:2], 0.125, ws)
    assert torch.all(out[2:] == 3.0) and torch.all(lse[2:] == 3.0)


def test_nan_in_a_live_row_stays_in_its_head(S):
    f = Filled(S, "bf16", [40, 40], 2, 64, 16, seed=13)
    f.cache.v[f.table[0, 1].item(), 1, 3, 5] = float("nan")
    q = _q(2, 4, 64, 5)
    ws = S.make_attn_workspace(f.cache, 4)
    out = f64(S.attn_decode(q, f.cache, f.table, f.seq_lens, ws))
    assert np.all(np.isnan(out[0, 2:, 5]))
    out[0, 2:, 5] = 0
    assert np.all(np.isfinite(out))


@pytest.mark.parametrize("hidden", [40, 1000, 9000, 9999])
def test_scores_of_minus_infinity_have_no_weight(S, hidden):
    # the first `hidden` keys are -infinity in a dim where q is positive: whole tiles,
    # warps' runs and CTAs' parts of no weight; a second sequence has nothing else
    f = Filled(S, "bf16", [10000, 70], 2, 64, 16, seed=hidden)
    pages = f.table.long().cpu()
    for b, n in ((0, hidden), (1, 70)):
        t = torch.arange(n)
        f.cache.k[pages[b, t // 16].cuda(), :, (t % 16).cuda(), 5] = float("-inf")
        f.k[b][:n, :, 5] = -np.inf
    q = _q(2, 4, 64, 8)
    q[:, :, 5] = 1.5
    ws = S.make_attn_workspace(f.cache, 4)
    lse = torch.zeros(2, 4, device="cuda")
    out = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, lse=lse)
    assert S.read_status(ws) == S.OK
    assert torch.isnan(out[1]).all() and torch.equal(lse[1], torch.full_like(lse[1], float("-inf")))
    # the sequence as if it began behind them
    g = Filled.__new__(Filled)
    g.kind, g.lens, g.heads, g.dim = f.kind, [10000 - hidden], f.heads, f.dim
    g.k, g.v = [f.k[0][hidden:]], [f.v[0][hidden:]]
    g.check(S, q[:1], out[:1], lse[:1], 64 ** -0.5, ws)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_bad_pages_are_reported_and_skipped(S, kind):
    f = Filled(S, kind, [40, 40, 40], 2, 64, 16, seed=14)
    q = _q(3, 4, 64, 6)
    ws = S.make_attn_workspace(f.cache, 4)
    good = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)
    assert S.read_status(ws) == S.OK
    for bad in (-1, f.n_pages, 1 << 30, -(1 << 31)):
        t = f.table.clone()
        t[1, 1] = bad
        out = S.attn_decode(q, f.cache, t, f.seq_lens, ws)
        assert S.read_status(ws) == S.ERR_DEVICE_CHECK
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    out = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)       # and the next call is clean
    assert S.read_status(ws) == S.OK and torch.equal(out, good)


def test_bad_lengths_are_reported_and_cut(S):
    f = Filled(S, "int8", [48, 48, 48], 2, 64, 16, seed=15)
    q = _q(3, 4, 64, 7)
    ws = S.make_attn_workspace(f.cache, 4)
    good = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)
    assert S.read_status(ws) == S.OK
    for bad in (-1, 49, 2147483647, -2147483648):
        n = f.seq_lens.clone()
        n[1] = bad
        out = S.attn_decode(q, f.cache, f.table, n, ws)
        assert S.read_status(ws) == S.ERR_DEVICE_CHECK
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


def test_same_result_every_time_and_in_a_shared_workspace(S):
    f = Filled(S, "int4", [1000, 3, 500], 2, 128, 16, seed=16)
    g = Filled(S, "int4", [64] * 40, 2, 128, 16, seed=17)
    q, out, lse, ws = _run(S, f, 4, seed=11)
    q2, out2, lse2, _ = _run(S, g, 4, seed=12, ws=ws)
    for _ in range(5):
        a = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)
        b = S.attn_decode(q2, g.cache, g.table, g.seq_lens, ws)
        assert torch.equal(a, out) and torch.equal(b, out2)


def test_caches_of_several_shapes_take_turns_in_a_workspace(S):
    shapes = [("bf16", 256, 4), ("int8", 128, 2), ("bf16", 64, 16), ("int4", 256, 8)]
    filled = [(Filled(S, kind, [9000, 3, 4000], 2, dim, 64, seed=i), group)
              for i, (kind, dim, group) in enumerate(shapes)]
    ws = max((S.make_attn_workspace(f.cache, 2 * group) for f, group in filled), key=torch.numel)
    for _ in range(2):
        for f, group in filled:
            _run(S, f, group, seed=9, ws=ws)


def test_graphs_that_share_a_workspace_follow_the_lengths(S):
    f = Filled(S, "bf16", [700, 32, 17], 2, 128, 16, seed=18)
    q = _q(3, 8, 128, 9)
    ws = S.make_attn_workspace(f.cache, 8)
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for o in outs:
            S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, out=o)
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, out=o)
            graphs.append(g)
    torch.cuda.synchronize()
    for lens in ([700, 32, 17], [13, 0, 16], [1, 32, 0], [699, 17, 2]):
        f.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        whole = f.lens, f.k, f.v
        f.lens, f.k, f.v = lens, [k[:n] for k, n in zip(f.k, lens)], [v[:n] for v, n in zip(f.v, lens)]
        for g, o in zip(graphs, outs):
            o.fill_(9.0)
            g.replay()
            f.check(S, q, o, None, 128 ** -0.5, ws)
        f.lens, f.k, f.v = whole


def test_on_another_stream(S):
    f = Filled(S, "int8", [300, 90], 2, 64, 16, seed=19)
    q = _q(2, 4, 64, 10)
    ws = S.make_attn_workspace(f.cache, 4)
    want = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    # two calls at once, a workspace each
    ws2 = S.make_attn_workspace(f.cache, 4)
    torch.cuda.synchronize()
    a = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws, stream=st)
    b = S.attn_decode(q, f.cache, f.table, f.seq_lens, ws2)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_offsets_past_32_bits(S):
    # 5 GiB of pages on each side; the sequence lies in the last ones
    n_pages, page, heads, dim = 40960, 64, 8, 128
    k = torch.empty((n_pages, heads, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() * 2 > 1 << 32
    f = Filled(S, "bf16", [200], heads, dim, page, seed=20, extra_pages=0)
    order = torch.tensor([n_pages - 1, n_pages - 4, 33000, 36000], device="cuda")
    for i, p in enumerate(order.tolist()):
        k[p].copy_(f.cache.k[f.table[0, i].item()])
        v[p].copy_(f.cache.v[f.table[0, i].item()])
    f.cache = S.kv_cache_from_parts(k, v)
    f.table[0, :4] = order.to(torch.int32)
    _run(S, f, 2, seed=13)


def test_binding_refusals(S):
    f = Filled(S, "int8", [20, 3], 2, 64, 16, seed=21)
    q, ws = _q(2, 4, 64, 1), S.make_attn_workspace(f.cache, 4)
    ok = (q, f.cache, f.table, f.seq_lens, ws)
    S.attn_decode(*ok)
    for i, bad in ((0, q.float()), (0, q.transpose(0, 1)), (0, q[:, :, ::2]), (2, f.table.long()), (2, f.table[:1]),
                   (3, f.seq_lens.long()), (3, f.seq_lens[:1]), (0, q.cpu()), (3, f.seq_lens.cpu()), (4, ws.cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            S.attn_decode(*args)
    with pytest.raises(S.SpearError):
        S.attn_decode(_q(2, 3, 64, 1), *ok[1:])                      # 3 heads over 2
    with pytest.raises(S.SpearError):
        S.attn_decode(*ok[:4], ws[:128])
    with pytest.raises(S.SpearError):
        S.attn_decode(*ok, scale=float("nan"))
    with pytest.raises(S.SpearError):
        S.attn_decode(*ok, out=q)
    with pytest.raises(ValueError):
        S.attn_decode(*ok, lse=torch.empty((2, 4), device="cuda", dtype=torch.float64))
    with pytest.raises(S.SpearError):
        S.make_attn_workspace(f.cache, 5)
    empty = S.attn_decode(q[:0], f.cache, f.table[:0], f.seq_lens[:0], ws)
    assert empty.shape == (0, 4, 64)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_pages_shared_between_sequences_and_repeated_in_one(S, kind):
    f = Filled(S, kind, [640, 640, 640], 2, 64, 32, seed=12)
    f.table[1] = f.table[0]                       # a second reader of the same tokens
    f.k[1], f.v[1] = f.k[0], f.v[0]
    f.table[2, 1:] = f.table[2, :1]               # one page for all of a sequence
    f.k[2], f.v[2] = (np.concatenate([t[2][:32]] * 20) for t in (f.k, f.v))
    q, out, _, ws = _run(S, f, 3, seed=13)
    same = q.clone()
    same[1] = q[0]
    again = S.attn_decode(same, f.cache, f.table, f.seq_lens, ws)
    assert torch.equal(again[0], out[0]) and torch.equal(again[2], out[2])


def test_two_calls_at_once_on_one_cache(S):
    f = Filled(S, "int8", [5000, 0, 37, 2100], 2, 128, 16, seed=14)
    qs = [_q(4, 8, 128, seed) for seed in (15, 16)]
    wss = [S.make_attn_workspace(f.cache, 8) for _ in qs]
    want = [S.attn_decode(q, f.cache, f.table, f.seq_lens, ws) for q, ws in zip(qs, wss)]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(S.attn_decode(qs[i], f.cache, f.table, f.seq_lens, wss[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert S.read_status(wss[i]) == S.OK
        assert all(torch.equal(g, want[i]) for g in got[i])
