"""Token steps of a small decoder through the library (linears, cache, attention,
norms together): every call against the float64 oracle on its own inputs, the
wiring between the calls, captured and replayed steps against eager ones."""
import numpy as np
import pytest
import torch

from oracle import spear_oracle as O
from tests.decoder_cases import Filled, bf16_tensor, f64
from tests.test_gpu_block_norm import _check as check_norm
from w4_gemm_gated_b200 import synth

pytestmark = pytest.mark.gpu

WIDTH, FF, HEAD, N_Q = 512, 1024, 64, 8
SHAPES = [(WIDTH, N_Q * HEAD), (WIDTH, 256), (WIDTH, 256), (N_Q * HEAD, WIDTH), (WIDTH, FF), (WIDTH, FF), (FF, WIDTH)]
N_KV = 256 // HEAD   # keys and values of a linear as narrow as the layer takes


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4_gemm_gated_b200 import build
    build.build()
    from w4_gemm_gated_b200 import spear
    return spear


def _bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _model(S, n_layers):
    mats, layers, norms = [], [], []
    rng = np.random.default_rng(5)
    for l in range(n_layers):
        row_m, row_l = [], []
        for proj, (K, N) in enumerate(SHAPES):
            ec = l == 0
            L = synth.make_layer(1, K, N, 16 if ec else 0, b_g=-1.0, seed=synth.stack_layer_seed(9, l, proj), w_std=0.05)
            q, s = O.quantize_rtn(L.W, 0)
            row_m.append((q, s, L.A, L.B, L.w_g, L.b_g))
            row_l.append(S.prepare_layer(torch.from_numpy(L.W).cuda(), 0, _bf16(L.A) if ec else None,
                                         _bf16(L.B) if ec else None, _bf16(L.w_g) if ec else None, L.b_g))
        mats.append(row_m)
        layers.append(row_l)
        norms.append(tuple(bf16_tensor(1 + 0.2 * rng.standard_normal(WIDTH)) for _ in range(2)))
    return mats, layers, norms


class _Recorder:
    """The binding, with the inputs and outputs of the calls of a step kept."""

    def __init__(self, S):
        self.S, self.calls = S, []

    def __getattr__(self, name):
        fn = getattr(self.S, name)
        if name not in ("forward", "kv_write", "attn_decode", "block_norm"):
            return fn

        def call(*args, **kw):
            out = fn(*args, **kw)
            self.calls.append((name, args, kw, out))
            return out

        return call


class _Held:
    """What the oracle says that a layer's cache holds (as Filled holds it)."""

    def __init__(self, kind, n_seqs):
        self.kind, self.dim, self.heads = kind, HEAD, N_KV
        self.k, self.v = ([np.zeros((0, N_KV, HEAD)) for _ in range(n_seqs)] for _ in range(2))

    def add(self, b, k, v):
        for held, x in ((self.k, k), (self.v, v)):
            x = x.reshape(1, N_KV, HEAD)
            held[b] = np.concatenate([held[b], x if self.kind == "bf16" else O.kv_values(*O.kv_quantize(x, self.kind))])
        self.lens = [len(t) for t in self.k]


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_every_call_of_a_step_against_the_oracle(S, monkeypatch, kind):
    """Each call's outputs within its own bound of the oracle's for the inputs that
    it got, and each gets what the one before it made."""
    from w4_gemm_gated_b200 import decoder
    n_seqs, steps = 3, 18
    mats, layers, norms = _model(S, 2)
    state = decoder.make_state(layers, n_seqs, 64, kind={"bf16": S.KV_BF16, "int8": S.KV_INT8, "int4": S.KV_INT4}[kind],
                               head_dim=HEAD)
    perm = torch.randperm(state.page_table.numel(), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    state.page_table.copy_(perm.view_as(state.page_table))
    held = [_Held(kind, n_seqs) for _ in layers]
    rec = _Recorder(S)
    monkeypatch.setattr(decoder, "S", rec)
    rng = np.random.default_rng(3)
    for t in range(steps):
        x = bf16_tensor(rng.standard_normal((n_seqs, WIDTH)))
        decoder.advance(state)
        late = t < 5                    # the last sequence starts late: its slot is skipped, its length 0
        if late:
            state.slots[2], state.seq_lens[2] = -1, 0
        rec.calls.clear()
        out = decoder.step(layers, x, state, norms=norms)
        assert decoder.status(state) == S.OK
        calls = iter(rec.calls)

        def norm_call(x, y, w, last=False):
            name, args, kw, got = next(calls)
            assert name == "block_norm" and args[0] is x and (y is None or args[1] is y) and kw["pre_weight"] is w
            tensors = {"x": x, "y": y if y is not None else torch.zeros_like(x), "post_weight": None, "gate": None,
                       "pre_weight": w}
            check_norm(tensors, got[0] if y is not None else None, got[1], 1.0, 1.0 if y is not None else 0.0, 1e-6)
            assert (got[1] is None) == last
            return got

        def linear(layer, mat, x):
            name, args, _, got = next(calls)
            assert name == "forward" and args[0] is layer and (x is None or args[1] is x)
            q, s, A, B, w_g, b_g = mat
            y, _ = O.linear(O.f32_to_bf16_bits_rne(f64(args[1]).astype(np.float32)), q, s, 0, A, B, w_g, b_g)
            assert np.max(np.abs(f64(got) - y)) <= 1e-2 * np.max(np.abs(y))     # the layer's stated bound
            return args[1], got

        _, h = norm_call(x, None, norms[0][0])
        for i, (row, mat) in enumerate(zip(layers, mats)):
            q, k, v = (linear(row[p], mat[p], h)[1] for p in range(3))
            name, args, _, _ = next(calls)
            assert name == "kv_write" and args[0] is state.caches[i] and args[1] is k and args[2] is v
            for b in range(n_seqs - late):
                held[i].add(b, f64(k)[b], f64(v)[b])
            name, args, _, a = next(calls)
            assert name == "attn_decode" and args[0] is q and args[1] is state.caches[i]
            want, _, tol, _ = Filled.expected(held[i], f64(q).reshape(n_seqs, N_Q, HEAD), HEAD ** -0.5)
            assert np.all(np.abs(f64(a).reshape(want.shape) - want) <= tol), (t, i)
            x, h = norm_call(x, linear(row[3], mat[3], a)[1], norms[i][1])
            gate, up = linear(row[4], mat[4], h)[1].float(), linear(row[5], mat[5], h)[1].float()
            act, y = linear(row[6], mat[6], None)
            assert torch.equal(act, (gate * torch.sigmoid(gate) * up).to(torch.bfloat16))
            last = i + 1 == len(layers)
            x, h = norm_call(x, y, None if last else norms[i + 1][0], last)
        assert x is out and next(calls, None) is None
    # and the caches hold, bit for bit, what the oracle says
    for cache, want in zip(state.caches, held):
        for b in range(n_seqs):
            at = torch.arange(want.lens[b], device="cuda")
            slots = state.page_table[b][at // cache.page_size] * cache.page_size + (at % cache.page_size).to(torch.int32)
            for got, values in zip(S.kv_read(cache, slots, state.attn_ws), (want.k[b], want.v[b])):
                assert torch.equal(got, bf16_tensor(values))


def test_captured_steps_follow_the_state(S):
    from w4_gemm_gated_b200 import decoder
    _, layers, norms = _model(S, 2)
    eager, replayed = (decoder.make_state(layers, 4, 48, kind=S.KV_INT4, head_dim=HEAD) for _ in range(2))
    rng = np.random.default_rng(4)
    x = torch.empty((4, WIDTH), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        decoder.advance(replayed)
        decoder.step(layers, x, replayed, norms=norms)
        replayed.seq_lens.zero_()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            decoder.advance(replayed)
            out = decoder.step(layers, x, replayed, norms=norms)
    torch.cuda.synchronize()
    for t in range(40):
        x.copy_(bf16_tensor(rng.standard_normal((4, WIDTH))))
        torch.cuda.synchronize()
        decoder.advance(eager)
        want = decoder.step(layers, x, eager, norms=norms)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), t
    assert decoder.status(eager) == S.OK and decoder.status(replayed) == S.OK
    assert torch.equal(eager.caches[1].k, replayed.caches[1].k)


def test_rotation_is_applied_before_the_cache(S):
    from w4_gemm_gated_b200 import decoder
    _, layers, _ = _model(S, 1)
    state = decoder.make_state(layers, 2, 16, kind=S.KV_BF16, head_dim=HEAD)
    x = bf16_tensor(np.random.default_rng(6).standard_normal((2, WIDTH)))
    decoder.advance(state)
    seen = []

    def rotate(q, k):
        seen.append((q, k))
        return -q, -k

    decoder.step(layers, x, state, rotate=rotate)
    back, _ = S.kv_read(state.caches[0], state.slots, state.attn_ws)
    assert torch.equal(back.view(2, -1), -seen[0][1]) and seen[0][0].shape == (2, N_Q * HEAD)


def test_a_step_past_the_last_page_is_reported(S):
    from w4_gemm_gated_b200 import decoder
    _, layers, _ = _model(S, 1)
    state = decoder.make_state(layers, 2, 16, kind=S.KV_INT8, head_dim=HEAD)
    state.seq_lens.copy_(torch.tensor([15, 3], dtype=torch.int32))
    x = bf16_tensor(np.random.default_rng(7).standard_normal((2, WIDTH)))
    decoder.advance(state)
    decoder.step(layers, x, state)
    assert decoder.status(state) == S.OK
    held = state.caches[0].k.clone()
    decoder.advance(state)                     # the first sequence's page is full
    assert state.slots.tolist() == [-1, 16 + 4]
    decoder.step(layers, x, state)
    assert decoder.status(state) == S.ERR_DEVICE_CHECK
    assert torch.equal(state.caches[0].k[0], held[0]) and not torch.equal(state.caches[0].k[1], held[1])
