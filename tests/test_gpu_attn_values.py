"""Attention over the paged cache where values are unlike one another: heavy
tokens of no value beside light ones, values of every magnitude, and the
output's precision over each cache kind."""
import numpy as np
import pytest
import torch

from tests.decoder_cases import HALF, Filled, bf16_tensor, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


def _close(f, q, got):
    """got within what 32 bits and two bf16 parts a weight leave of the 64-bit output.

    The weights: the score's error (as Filled.expected has it), the exponential's
    2^-20, the two parts' 2^-17 and the product with the value's scale, 2^-24.  The
    sums: as many roundings as tokens at most, of partial sums of the magnitudes, and
    16 more where parts are joined.  Then the output's own rounding."""
    q64 = f64(q)
    want, _, _, _ = f.expected(q64, f.dim ** -0.5)
    G = q64.shape[1] // f.heads
    for b, n in enumerate(f.lens):
        if n == 0:
            assert np.all(got[b] == 0)
            continue
        kk = np.abs(f.k[b])
        sum_q = np.sum(np.abs(q64[b]), axis=-1)
        if f.kind == "bf16":
            ds = np.max(np.sum(np.abs(q64[b]) * np.repeat(kk.max(axis=0), G, axis=0), axis=-1)) * (f.dim + 8) * 2.0 ** -24
        else:
            top, Q = (255, 127) if f.kind == "int8" else (15, 7)
            s = np.repeat(kk.max(axis=(0, 2)), G) / Q * 1.01
            ds = np.max(sum_q * s) * 2 * top * (f.dim / 16 + 3) * 2.0 ** -23
        ds *= f.dim ** -0.5
        for h in range(q64.shape[1]):
            score = (f.k[b][:, h // G] @ q64[b, h]) * f.dim ** -0.5
            p = np.exp(score - score.max())
            pv = (p / p.sum()) @ np.abs(f.v[b][:, h // G])
            before = (2.0 ** -17 + 2 * ds + 2.0 ** -20 + (min(n, 4096) + 17) * 2.0 ** -24) * pv
            off = np.abs(got[b, h] - want[b, h]) / (HALF * np.abs(want[b, h]) + (1 + HALF) * before + 1e-37)
            assert np.all(off <= 1.0), f"sequence {b} head {h}: {np.max(off):.2f} of the bound"


def _towards(f, token, nats, group, seed):
    """q whose score with the token is about nats above the others' of every sequence."""
    rng = np.random.default_rng(seed)
    q = rng.standard_normal((len(f.lens), f.heads * group, f.dim))
    for b, n in enumerate(f.lens):
        if n > token:
            k = np.repeat(f.k[b][token], group, axis=0)
            size = np.sum(k * k, axis=-1, keepdims=True)
            q[b] += k * (nats * f.dim ** 0.5 - np.sum(q[b] * k, axis=-1, keepdims=True)) / size
    return q


def _silence(f, tokens):
    """Values of no size at these tokens of every sequence, as kv_write stores them: scale 1, codes 0."""
    for b, n in enumerate(f.lens):
        t = np.array([i for i in tokens if i < n], dtype=np.int64)
        if not len(t):
            continue
        f.v[b][t] = 0
        page = f.table[b][torch.from_numpy(t // f.page).cuda()].long()
        off = torch.from_numpy(t % f.page).cuda()
        f.cache.v[page, :, off] = 0x88 if f.kind == "int4" else 0
        if f.kind != "bf16":
            f.cache.v_scales[page, :, off] = 1.0


@pytest.mark.parametrize("kind", ["int8", "int4", "bf16"])
@pytest.mark.parametrize("nats,size", [(15, 0.02), (12, 1e-3), (30, 1e-3), (45, 0.5)])
@pytest.mark.parametrize("group", [1, 4, 12])
def test_a_heavy_token_of_no_value_leaves_the_others_theirs(S, kind, nats, size, group):
    f = Filled(S, kind, [512, 40, 3, 2500], 2, 128, 16, seed=group, spread=size)
    _silence(f, [0, 33])
    q = bf16_tensor(_towards(f, 0, nats, group, seed=nats))
    ws = S.make_attn_workspace(f.cache, 2 * group)
    got = f64(S.attn_decode(q, f.cache, f.table, f.seq_lens, ws))
    assert S.read_status(ws) == S.OK
    _close(f, q, got)


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_mostly_padding_of_no_value(S, kind):
    f = Filled(S, kind, [700, 64], 2, 64, 16, seed=3, spread=4e-4)
    _silence(f, [t for t in range(700) if t % 7])
    q = bf16_tensor(_towards(f, 5, 10, 4, seed=4))
    ws = S.make_attn_workspace(f.cache, 8)
    _close(f, q, f64(S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)))


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("order", [1, -1])
def test_scales_of_every_magnitude_in_a_sequence(S, kind, order):
    # values from 2^-12 to 2^12, rising or falling along the sequence, the heaviest token at an end
    f = Filled(S, kind, [400], 2, 128, 32, seed=6)
    power = np.linspace(-12, 12, 400).astype(np.int64)[::order]
    page = f.table[0][torch.arange(400, device="cuda") // 32].long()
    off = torch.arange(400, device="cuda") % 32
    codes = np.rint(f.v[0] / f64(f.cache.v_scales[page, :, off])[:, :, None])
    by = torch.from_numpy(np.exp2(power)).to(torch.float16).cuda()
    f.cache.v_scales[page, :, off] = f.cache.v_scales[page, :, off] * by[:, None]
    f.v[0] = codes * f64(f.cache.v_scales[page, :, off])[:, :, None]
    for token in (0, 399):
        q = bf16_tensor(_towards(f, token, 14, 2, seed=7))
        ws = S.make_attn_workspace(f.cache, 4)
        _close(f, q, f64(S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)))


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 16])
def test_outputs_to_the_precision_of_32_bits(S, kind, dim, group):
    f = Filled(S, kind, [1, 0, 16, 33, 450], 2, dim, 16, seed=dim + group)
    q = bf16_tensor(np.random.default_rng(dim).standard_normal((5, 2 * group, dim)))
    ws = S.make_attn_workspace(f.cache, 2 * group)
    _close(f, q, f64(S.attn_decode(q, f.cache, f.table, f.seq_lens, ws)))


INF = float("inf")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 12])
def test_infinite_values_are_infinite_outputs(S, dim, group):
    f = Filled(S, "bf16", [1, 2, 33, 700, 4000], 2, dim, 16, seed=dim + group)
    rng = np.random.default_rng(8)
    want = {}
    for b, n in enumerate(f.lens):
        # a dim each of +, -, both, NaN, and + twice, at tokens of their own
        for d, what in ((1, (INF,)), (6, (-INF,)), (dim - 3, (INF, -INF)), (dim // 2, (float("nan"),)), (17, (INF, INF))):
            tokens = rng.permutation(n)[:len(what)]
            what = what[:len(tokens)]
            for g in range(2):
                for t, x in zip(tokens, what):
                    f.cache.v[f.table[b, t // 16].long(), g, t % 16, d] = x
                f.v[b][tokens, g, d] = 0.0
            want[b, d] = sum(what)
    q = bf16_tensor(rng.standard_normal((5, 2 * group, dim)))
    ws = S.make_attn_workspace(f.cache, 2 * group)
    got = f64(S.attn_decode(q, f.cache, f.table, f.seq_lens, ws))
    for (b, d), x in want.items():
        assert np.array_equal(got[b, :, d], np.full(2 * group, x), equal_nan=True), (b, d, got[b, :, d])
        got[b, :, d] = 0.0
        f.v[b][:, :, d] = 0.0
    _close(f, q, got)      # the other dims, as if nothing lay beside them


def test_an_infinite_value_without_weight_and_behind_the_end(S):
    # its key is -infinity: 0 times infinity; behind a sequence's end nothing is read
    f = Filled(S, "bf16", [50, 20], 1, 64, 16, seed=9)
    f.cache.v[f.table[0, 2].long(), 0, 3, 7] = INF        # token 35
    f.cache.k[f.table[0, 2].long(), 0, 3, 5] = -INF
    f.cache.v[f.table[1, 1].long(), 0, 4, 7] = INF        # token 20 of 20
    q = bf16_tensor(np.random.default_rng(10).standard_normal((2, 2, 64)))
    q[:, :, 5] = 1.0
    ws = S.make_attn_workspace(f.cache, 2)
    got = f64(S.attn_decode(q, f.cache, f.table, f.seq_lens, ws))
    assert np.all(np.isnan(got[0, :, 7])) and np.isfinite(got).sum() == got.size - 2
