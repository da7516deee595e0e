"""Shared pieces of the decoder-step GPU tests: caches filled from the oracle's
codes, with every place that no call may use poisoned, and error bounds."""
import numpy as np
import torch

from oracle import spear_oracle as O

HALF = float(torch.finfo(torch.bfloat16).eps) / 2      # a rounding to bf16, relative to the value
KINDS = {"bf16": 0, "int8": 1, "int4": 2}
DT = {"bf16": torch.bfloat16, "int8": torch.int8, "int4": torch.uint8}


def bf16_tensor(v, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16).to(device)


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16_values(rng, *shape, scale=1.0):
    """float64 array of values that bf16 holds."""
    v = (rng.standard_normal(shape) * scale).astype(np.float32)
    return O.bf16_to_f64(O.f32_to_bf16_bits_rne(v))


class Filled:
    """A cache of sequences of the given lengths over shuffled pages.  k, v: lists
    of L x G x D float64 values as the cache holds them."""

    def __init__(self, S, kind, lens, heads, dim, page, seed, spread=1.0, extra_pages=2, apart=False, max_pages=None):
        rng = np.random.default_rng(seed)
        self.kind, self.lens, self.page, self.heads, self.dim = kind, lens, page, heads, dim
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + extra_pages
        width = dim // 2 if kind == "int4" else dim
        order = rng.permutation(n_pages)
        self.width = max_pages or max(1, max(need))
        # entries past a sequence's length are never read: numbers of no page
        table = rng.choice([-1, 1 << 30, -(1 << 31), n_pages], size=(len(lens), self.width)).astype(np.int32)
        codes = {s: np.zeros((n_pages, heads, page, width), dtype=np.float32) for s in "kv"}
        scales = {s: np.full((n_pages, heads, page), np.nan, dtype=np.float16) for s in "kv"}
        if kind == "bf16":
            for s in "kv":
                codes[s][:] = np.where(rng.random(codes[s].shape) < 0.5, np.nan, np.inf)
        else:
            for s in "kv":
                codes[s][:] = rng.integers(0, 255, codes[s].shape) - (128 if kind == "int8" else 0)
        self.k, self.v, at = [], [], 0
        for b, n in enumerate(lens):
            pages = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = pages
            for s, keep in (("k", self.k), ("v", self.v)):
                x = bf16_values(rng, n, heads, dim, scale=spread)
                if kind == "bf16":
                    stored, val, sc = x, x, None
                else:
                    q, sc = O.kv_quantize(x, kind)
                    val = O.kv_values(q, sc)
                    stored = q if kind == "int8" else O.kv_pack4(q)
                t = np.arange(n)
                if n:
                    codes[s][pages[t // page], :, t % page] = stored
                    if sc is not None:
                        scales[s][pages[t // page], :, t % page] = sc
                keep.append(val)
        self.n_pages = n_pages

        def put(a, dtype):
            t = torch.from_numpy(a)
            t = t.to(dtype) if dtype == torch.bfloat16 or dtype == torch.float16 else t.to(torch.int16).to(dtype)
            if not apart:
                return t.cuda()
            # pages inside a wider allocation, with poison between them
            flat = t.reshape(n_pages, -1)
            gap = torch.full((n_pages, 64), float("nan") if t.is_floating_point() else 77).to(dtype)
            whole = torch.cat([flat, gap], dim=1).cuda()
            return torch.as_strided(whole, t.shape, (whole.stride(0), t[0].numel() // heads, t.stride(2),
                                                     *((1,) if t.dim() == 4 else ())))

        parts = [put(codes[s], DT[kind]) for s in "kv"]
        if kind != "bf16":
            parts += [put(scales[s], torch.float16) for s in "kv"]
        self.cache = S.kv_cache_from_parts(*parts)
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def expected(self, q, scale):
        """out, lse and the bounds of both for q (n x H x D float64)."""
        outs, lses, tol_o, tol_l = [], [], [], []
        D, H = self.dim, q.shape[1]
        G = H // self.heads
        for b, n in enumerate(self.lens):
            o, l, p = O.attend(q[b], self.k[b], self.v[b], scale)
            # The score's error.  bf16: a sum of D products in 32 bits and its scalings.
            # Codes enter as u = c + 128 or c + 8, and the sum starts at minus what that
            # adds: terms up to 255 s |q| (15 s |q|) and a start of up to 128 (8) of them,
            # in D / 16 products whose sums are each off by a step of 32 bits (2^-23) at
            # most, and three scalings.  No scale s is above max|k| / Q (1 + 2^-11).
            ds = 0.0
            if n:
                sum_q = np.sum(np.abs(q[b]), axis=-1)                              # H
                if self.kind == "bf16":
                    kk = np.repeat(np.abs(self.k[b]).max(axis=0), G, axis=0)       # H x D
                    ds = np.max(np.sum(np.abs(q[b]) * kk, axis=-1)) * (D + 8) * 2.0 ** -24
                else:
                    top, Q = (255, 127) if self.kind == "int8" else (15, 7)
                    s = np.repeat(np.abs(self.k[b]).max(axis=(0, 2)), G) / Q * 1.01    # H
                    ds = np.max(sum_q * s) * 2 * top * (D / 16 + 3) * 2.0 ** -23
                ds *= abs(scale)
            # Weights off by the score's error and the exponential's (2^-20), each rounded
            # to two bf16 parts (2^-17), or with its value's scale to fp16 (2^-11, and
            # where it is under 2^-25 of the largest, to 2^-36 of that); products summed in
            # 32 bits (as many roundings as tokens at most, of partial sums of the magnitudes).
            pv = np.stack([p[h] @ np.abs(self.v[b][:, h // G]) for h in range(H)]) if n else np.zeros((H, D))
            rounding, lost = 2.0 ** -17, 0.0
            if self.kind != "bf16":
                rounding, lost = 2.0 ** -11, n * 2.0 ** -36 * (np.abs(self.v[b]).max() if n else 0.0)
            tol_o.append(HALF * np.abs(o) + (rounding + 2 * ds + 2.0 ** -20 + min(n + 16, 4096) * 2.0 ** -24) * pv + lost
                         + 1e-30)
            tol_l.append(np.full(H, ds + 2.0 ** -20) + 2.0 ** -22 * np.where(np.isfinite(l), np.abs(l), 0) +
                         (n + 16) * 2.0 ** -24)
            outs.append(o)
            lses.append(l)
        return np.stack(outs), np.stack(lses), np.stack(tol_o), np.stack(tol_l)

    def check(self, S, q, out, lse, scale, ws):
        torch.cuda.synchronize()
        assert S.read_status(ws) == S.OK
        o, l, to, tl = self.expected(f64(q).reshape(len(self.lens), -1, self.dim), scale)
        got = f64(out).reshape(o.shape)
        assert np.all(np.isfinite(got))
        worst = np.max(np.abs(got - o) / to)
        assert worst <= 1.0, f"out off by {worst:.2f} of the bound"
        if lse is not None:
            gl = f64(lse)
            none = np.isinf(l)
            assert np.array_equal(gl[none], l[none])
            if (~none).any():
                worst = np.max(np.abs(gl[~none] - l[~none]) / tl[~none])
                assert worst <= 1.0, f"lse off by {worst:.2f} of the bound"
