"""Bytes that the cache, attention and norm calls must leave alone: guards around
every output and workspace, everything in a cache's allocation but the slots
written.  Once on the normal library, once in a child process on the
device-check build, whose checks of output stores, parts, counters and rows
must find nothing."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests.decoder_cases import Filled, bf16_tensor, f64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

GUARD = 4096     # bytes on each side
MARK = 0xA5

# kind, lengths, kv heads, head dim, page, query heads per kv head, longest table
ATTENTION = [
    ("bf16", [1, 0, 17], 2, 64, 16, 3, None),
    ("int8", [33, 700, 0, 5], 1, 128, 32, 13, None),
    ("int4", [90, 2500], 3, 256, 16, 1, None),
    ("bf16", [9000, 3], 2, 256, 64, 16, None),          # parts of several CTAs
    ("int8", [6400] * 18, 1, 128, 64, 4, None),         # joined in groups, two units in a CTA
    ("int4", [6000, 0, 1, 130], 1, 128, 64, 16, 1500),  # two products side by side
    ("int8", [5] * 400, 2, 64, 16, 1, None),            # more sequences than threads
]


class Guarded:
    """A tensor between guard bytes."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.whole = torch.full((n + 2 * GUARD,), MARK, dtype=torch.uint8, device="cuda")
        self.t = self.whole[GUARD:GUARD + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.whole[:GUARD] == MARK).all() and (self.whole[-GUARD:] == MARK).all())


def _attention(S):
    found = []
    for i, (kind, lens, heads, dim, page, group, width) in enumerate(ATTENTION):
        f = Filled(S, kind, lens, heads, dim, page, seed=i, apart=True, max_pages=width)
        H, n = heads * group, len(lens)
        q = bf16_tensor(np.random.default_rng(i).standard_normal((n, H, dim)))
        ws = Guarded((S.attn_workspace_bytes(f.cache, H),), torch.uint8)
        assert S.F["spear_workspace_init"](ws.t.data_ptr(), ws.t.numel(), None) == S.OK
        out, lse = Guarded((n, H, dim), torch.bfloat16), Guarded((n, H), torch.float32)
        for _ in range(2):
            S.attn_decode(q, f.cache, f.table, f.seq_lens, ws.t, out=out.t, lse=lse.t)
        torch.cuda.synchronize()
        status = S.read_status(ws.t)
        f.check(S, q, out.t, lse.t, dim ** -0.5, ws.t)
        found.append({"case": str(ATTENTION[i])[:60], "status": status,
                      "guards": ws.intact() and out.intact() and lse.intact()})
    return found


def _cache(S):
    found = []
    for i, (kind, heads, dim, page, n) in enumerate([("BF16", 3, 64, 16, 37), ("INT8", 5, 128, 32, 1), ("INT4", 1, 256, 16, 70),
                                                     ("INT8", 7, 64, 16, 2000), ("INT4", 8, 128, 64, 1000)]):
        cache = S.make_kv_cache(getattr(S, "KV_" + kind), -(-n // page) + 3, page, heads, dim)
        parts = [t for t in (cache.k, cache.v, cache.k_scales, cache.v_scales) if t is not None]
        held = [Guarded(t.shape, t.dtype) for t in parts]
        cache = S.kv_cache_from_parts(*(g.t for g in held))
        rng = np.random.default_rng(i)
        k, v = (bf16_tensor(rng.standard_normal((n, heads, dim))) for _ in range(2))
        slots = rng.permutation(cache.n_pages * page)[:n]
        ws = Guarded((256,), torch.uint8)
        assert S.F["spear_workspace_init"](ws.t.data_ptr(), 256, None) == S.OK
        at = torch.from_numpy(slots.astype(np.int32)).cuda()
        S.kv_write(cache, k, v, at, ws.t)
        outs = [Guarded((n, heads, dim), torch.bfloat16) for _ in range(2)]
        S.kv_read(cache, at, ws.t, k_out=outs[0].t, v_out=outs[1].t)
        torch.cuda.synchronize()
        status = S.read_status(ws.t)
        free = np.setdiff1d(np.arange(cache.n_pages * page), slots)
        page_of, off = (torch.from_numpy(a).cuda() for a in (free // page, free % page))
        rest = all(bool((g.t[page_of, :, off].contiguous().view(torch.uint8) == MARK).all()) for g in held)
        near = all(np.all(np.abs(f64(o.t) - f64(x)) <= np.abs(f64(x)).max() * {"BF16": 0, "INT8": .01, "INT4": .1}[kind])
                   for o, x in zip(outs, (k, v)))
        found.append({"case": f"{kind} {heads} {dim} {page} {n}", "status": status, "near": near,
                      "guards": rest and ws.intact() and all(g.intact() for g in held + outs)})
    return found


def _norm(S):
    found = []
    for M, K in ((1, 8), (3, 264), (5, 4096), (2, 16384), (700, 1000)):
        rng = np.random.default_rng(K)
        x, y, gate = (bf16_tensor(rng.standard_normal((M, K))) for _ in range(3))
        w = bf16_tensor(rng.standard_normal(K))
        xo, h = (Guarded((M, K), torch.bfloat16) for _ in range(2))
        S.block_norm(x, y, pre_weight=w, post_weight=w, gate=gate, x_out=xo.t, h=h.t)
        torch.cuda.synchronize()
        found.append({"case": f"norm {M} {K}", "status": 0, "guards": xo.intact() and h.intact()})
    return found


def run_cases(S):
    return _attention(S) + _cache(S) + _norm(S)


def child_main():
    from w4_gemm_gated_b200 import spear as S
    print(json.dumps({"checks": int(S.F["spear_device_checks_enabled"]()), "cases": run_cases(S)}), flush=True)


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4_gemm_gated_b200 import build
    build.build()
    build.build(checked=True)
    from w4_gemm_gated_b200 import spear
    return spear


def _check(cases):
    for c in cases:
        assert c["status"] == 0 and c["guards"] and c.get("near", True), c


def test_guards_normal_build(S):
    _check(run_cases(S))


def test_guards_and_checks_of_the_device_check_build(S):
    env = dict(os.environ, SPEAR_DEVICE_CHECKS="1", PYTHONPATH=ROOT)
    proc = subprocess.run([sys.executable, "-c", "import tests.test_gpu_decoder_guards as t; t.child_main()"], cwd=ROOT,
                          env=env, capture_output=True, text=True, timeout=900)
    assert proc.returncode == 0, proc.stderr[-3000:]
    res = json.loads(proc.stdout.strip().splitlines()[-1])
    assert res["checks"] == 1
    _check(res["cases"])
