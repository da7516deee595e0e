"""Measured cases of the operators around the W4 linears of a decoder step: the
quantised key-value cache (write, read back), the attention of one new token
per sequence over its pages, and the norms around a block with its gate and
residual scale.

``run`` computes them in plain torch operations, in 32 bits and rounded once at
the end, or, where ``own`` is set, through the library's calls.  ``exact``
computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
LEVELS = {"int8": 127.0, "int4": 7.0}
BITS = {"bf16": 16, "int8": 8, "int4": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    attn = dict(op="attn")
    kv = dict(op="kv")
    norm = dict(op="norm")
    return [
        # one user's short chat: latency of a call that reads half a megabyte
        dict(attn, name="attn-one-short", kind="bf16", batch=1, heads=32, kv_heads=8, dim=128, page=16, longest=97),
        # an odd head group over 64-wide heads, a sequence of no tokens and one of a single token among them
        dict(attn, name="attn-odd-group", kind="int8", batch=7, heads=14, kv_heads=2, dim=64, page=64, longest=1001),
        # a small server's batch over an int8 cache
        dict(attn, name="attn-batch-int8", kind="int8", batch=16, heads=32, kv_heads=8, dim=128, page=16, longest=2048),
        # a full batch over a bf16 cache
        dict(attn, name="attn-batch-bf16", kind="bf16", batch=64, heads=32, kv_heads=8, dim=128, page=16, longest=4096),
        # 32 heads of 128 with keys and values of their own (the stack's 4096 x 4096 k and v), 4-bit cache
        dict(attn, name="attn-mha-int4", kind="int4", batch=32, heads=32, kv_heads=32, dim=128, page=32, longest=4099),
        # two users with whole books in the cache
        dict(attn, name="attn-long-bf16", kind="bf16", batch=2, heads=32, kv_heads=8, dim=128, page=64, longest=131072),
        # a decode step's sixteen new tokens, and the start of their prompts read back
        dict(kv, name="kv-append-int8", kind="int8", batch=16, kv_heads=8, dim=128, page=16, new=1, longest=40),
        # chunked prefill: the chunk is written, then the whole context is read back for its attention
        dict(kv, name="kv-chunk-int4", kind="int4", batch=4, kv_heads=32, dim=128, page=32, new=129, longest=2048),
        # the same for a full prefill batch
        dict(kv, name="kv-prefill-int8", kind="int8", batch=8, kv_heads=8, dim=128, page=16, new=1024, longest=8192),
        # the glue of one token of one user
        dict(norm, name="norm-one-token", rows=1, width=4096, post=False, gate="none", scales=False),
        # the stack's 256 tokens, norms on both sides of the block, a gate for each channel
        dict(norm, name="norm-stack", rows=256, width=4096, post=True, gate="channel", scales=True),
        # a full prefill with a gate for each token and channel
        dict(norm, name="norm-prefill", rows=8192, width=4096, post=True, gate="token", scales=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "attn", "kv", "norm"))
    if op == "norm":
        width = 8 * _log(rng, 16, 1792)
        rows = _log(rng, 1, max(1, 8192 * 4096 // width))
        return dict(op=op, rows=rows, width=width, post=rng.random() < 0.6,
                    gate=rng.choice(("none", "channel", "token")), scales=rng.random() < 0.5)
    kind = rng.choice(("bf16", "int8", "int4"))
    dim = rng.choice((64, 128, 128, 256))
    page = rng.choice((16, 32, 64, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 5, 8, 8, 16, 32))
    # tokens in all, so that no case moves more than the largest listed one
    most = 8e8 / (kv_heads * dim * BITS[kind] / 4) if op == "attn" else 1.2e8 / (kv_heads * dim * 4)
    batch = _log(rng, 1, 128)
    longest = _log(rng, 2, max(4, min(131072, most / batch)))
    if op == "attn":
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
        return dict(op=op, kind=kind, batch=batch, heads=group * kv_heads, kv_heads=kv_heads, dim=dim, page=page,
                    longest=longest)
    new = _log(rng, 1, longest)
    return dict(op=op, kind=kind, batch=batch, kv_heads=kv_heads, dim=dim, page=page, new=new, longest=longest)


def lengths(case):
    """The sequences' lengths: the longest, and others below it; in a batch of
    five or more, one of a single token and (attention) one of none."""
    rng = random.Random(case["longest"] * 1000 + case["batch"])
    n = [case["longest"]] + [rng.randint(max(1, case["longest"] // 8), case["longest"])
                             for _ in range(case["batch"] - 1)]
    if case["batch"] >= 5:
        n[2] = 1
        if case["op"] == "attn":
            n[4] = 0
    return n


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _random_pages(g, kind, n_pages, case, offset):
    """A cache's contents (codes, scales) as earlier writes left them."""
    heads, page, dim = case["kv_heads"], case["page"], case["dim"]
    if kind == "bf16":
        out = torch.empty((n_pages, heads, page, dim), dtype=torch.bfloat16, device=DEV)
        out.normal_(generator=g)
        return out.add_(offset), None
    # rows of N(offset, 1): the largest of them sets the scale
    spread = (3.0 if kind == "int8" else 2.5) + abs(offset)
    scale = (spread + torch.rand((n_pages, heads, page), generator=g, device=DEV)) / LEVELS[kind]
    scale = scale.to(torch.float16)
    most = int(LEVELS[kind])
    codes = torch.empty((n_pages, heads, page, dim), dtype=torch.float16, device=DEV).normal_(generator=g)
    codes = codes.add_(offset).div_(scale.unsqueeze(-1)).round_().clamp_(-most, most).to(torch.int8)
    return (codes if kind == "int8" else _nibbles(codes)), scale


def _nibbles(codes):
    u = (codes + 8).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        return _prepare_norm(case, g)
    lens = lengths(case)
    width = max(1, max(-(-n // case["page"]) for n in lens))
    n_pages = sum(-(-n // case["page"]) for n in lens) + 3   # a few that belong to nobody
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((case["batch"], width), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // case["page"])
        table[b, :k] = order[at:at + k]
        at += k
    st = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    st["k"], st["k_scale"] = _random_pages(g, case["kind"], n_pages, case, 0.25)
    st["v"], st["v_scale"] = _random_pages(g, case["kind"], n_pages, case, 0.0)
    if case["op"] == "attn":
        st["q"] = (_randn(g, case["batch"], case["heads"], case["dim"]) * 1.5).to(torch.bfloat16)
    else:
        news = [min(case["new"], n) for n in lens]
        seq = torch.cat([torch.full((n,), b, device=DEV) for b, n in enumerate(lens)])
        pos = torch.cat([torch.arange(n, device=DEV) for n in lens])
        slots = table[seq, pos // case["page"]] * case["page"] + (pos % case["page"]).to(torch.int32)
        fresh = torch.cat([torch.arange(n, device=DEV) >= n - k for n, k in zip(lens, news)])
        st["read"], st["write"] = slots, slots[fresh].contiguous()
        shape = (sum(news), case["kv_heads"], case["dim"])
        # keys with the few large channels that they have in earnest
        wide = 1.0 + 7.0 * (torch.rand((1, case["kv_heads"], case["dim"]), generator=g, device=DEV) < 0.02)
        st["new_k"] = (_randn(g, *shape) * wide).to(torch.bfloat16)
        st["new_v"] = _randn(g, *shape).to(torch.bfloat16)
    if own:
        from w4_gemm_gated_b200 import spear as S
        st["cache"] = S.kv_cache_from_parts(st["k"], st["v"], st["k_scale"], st["v_scale"])
        st["ws"] = S.make_attn_workspace(st["cache"], case.get("heads", case["kv_heads"]))
    return st


def _prepare_norm(case, g):
    rows, width = case["rows"], case["width"]
    st = {"case": case,
          "x": (_randn(g, rows, width) * 2).to(torch.bfloat16),
          "y": (_randn(g, rows, width) * 0.5).to(torch.bfloat16),
          "pre": (1 + 0.1 * _randn(g, width)).to(torch.bfloat16),
          "post": (1 + 0.1 * _randn(g, width)).to(torch.bfloat16) if case["post"] else None,
          "gate": None, "res": 0.75 if case["scales"] else 1.0, "blk": 1.25 if case["scales"] else 1.0}
    if case["gate"] != "none":
        n = 1 if case["gate"] == "channel" else rows
        st["gate"] = torch.rand((n, width), generator=g, device=DEV).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        from w4_gemm_gated_b200 import spear as S
        if op == "attn":
            return S.attn_decode(st["q"], st["cache"], st["table"], st["lens"], st["ws"])
        if op == "kv":
            S.kv_write(st["cache"], st["new_k"], st["new_v"], st["write"], st["ws"])
            return S.kv_read(st["cache"], st["read"], st["ws"])
        return S.block_norm(st["x"], st["y"], pre_weight=st["pre"], post_weight=st["post"], gate=st["gate"],
                            residual_scale=st["res"], block_scale=st["blk"], eps=EPS)
    if op == "attn":
        return _plain_attn(st)
    return _plain_kv(st) if op == "kv" else _plain_norm(st)


def _values(kind, codes, scale):
    """fp32 values of a cache's rows."""
    if kind == "bf16":
        return codes.float()
    if kind == "int4":
        codes = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float() - 8.0
    return codes.float() * scale.float().unsqueeze(-1)


def _plain_attn(st):
    c = st["case"]
    batch, heads, kv_heads, dim = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    pages = st["table"].long()

    def gathered(codes, scale):
        x = _values(c["kind"], codes[pages], None if scale is None else scale[pages])   # [B, pages, H, P, D]
        return x.transpose(1, 2).reshape(batch, kv_heads, -1, dim)

    q = st["q"].float().view(batch, kv_heads, heads // kv_heads, dim)
    s = (q @ gathered(st["k"], st["k_scale"]).transpose(-1, -2)) * (1.0 / math.sqrt(dim))
    live = torch.arange(s.shape[-1], device=DEV) < st["lens"].view(-1, 1, 1, 1)
    s = s.masked_fill(~live, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p @ gathered(st["v"], st["v_scale"])) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(batch, heads, dim).to(torch.bfloat16)


def _quantised(x, kind):
    """Codes and fp16 scales of rows of bf16 values: the quotients are of 32 bits by the operator's definition."""
    x = x.float()
    most = torch.full((), LEVELS[kind], device=DEV)
    s = (x.abs().amax(-1) / most).clamp(max=65504.0).to(torch.float16)
    none = s == 0
    s = torch.where(none, torch.ones_like(s), s)
    codes = torch.round(x / s.float().unsqueeze(-1)).clamp(-LEVELS[kind], LEVELS[kind])
    codes = torch.where(none.unsqueeze(-1), torch.zeros_like(codes), codes).to(torch.int8)
    return (codes if kind == "int8" else _nibbles(codes)), s


def _plain_kv(st):
    c = st["case"]
    page, off = (st["write"] // c["page"]).long(), (st["write"] % c["page"]).long()
    rpage, roff = (st["read"] // c["page"]).long(), (st["read"] % c["page"]).long()

    def one(codes, scale, new):
        if c["kind"] == "bf16":
            codes[page, :, off] = new
            return codes[rpage, :, roff]
        q, s = _quantised(new, c["kind"])
        codes[page, :, off] = q
        scale[page, :, off] = s
        return _values(c["kind"], codes[rpage, :, roff], scale[rpage, :, roff]).to(torch.bfloat16)

    return one(st["k"], st["k_scale"], st["new_k"]), one(st["v"], st["v_scale"], st["new_v"])


def _plain_norm(st):
    y = st["y"].float()
    if st["post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * st["post"].float()
    if st["gate"] is not None:
        y = y * st["gate"].float()
    x = st["x"].float() * st["res"] + y * st["blk"]
    h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["pre"].float()
    return x.to(torch.bfloat16), h.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(st)
    return _exact_kv(st) if case["op"] == "kv" else _exact_norm(st)


def _row64(kind, codes, scale):
    if kind == "bf16":
        return codes.double()
    if kind == "int8":
        return codes.double() * scale.double()[..., None]
    out = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=DEV)
    out[..., 0::2] = (codes % 16).double() - 8
    out[..., 1::2] = (codes // 16).double() - 8
    return out * scale.double()[..., None]


def _exact_attn(st):
    """Sequence by sequence and head by head."""
    c = st["case"]
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros((c["batch"], c["heads"], c["dim"]), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lengths(c)):
        if n == 0:
            continue
        at = torch.arange(n, device=DEV)
        page, off = st["table"][b][at // c["page"]].long(), at % c["page"]
        for h in range(c["kv_heads"]):
            ks = None if st["k_scale"] is None else st["k_scale"][page, h, off]
            vs = None if st["v_scale"] is None else st["v_scale"][page, h, off]
            k, v = _row64(c["kind"], st["k"][page, h, off], ks), _row64(c["kind"], st["v"][page, h, off], vs)
            rows = slice(h * group, (h + 1) * group)
            s = torch.einsum("gd,td->gt", st["q"][b, rows].double(), k) / math.sqrt(c["dim"])
            out[b, rows] = torch.softmax(s, -1) @ v
    return out


def _exact_kv(st):
    c = st["case"]
    where = {int(s): i for i, s in enumerate(st["write"].tolist())}
    pick = torch.tensor([where.get(int(s), -1) for s in st["read"].tolist()], device=DEV)
    fresh = pick >= 0
    read = st["read"].long()
    page, off = read // c["page"], read % c["page"]
    got = []
    for codes, scale, new in ((st["k"], st["k_scale"], st["new_k"]), (st["v"], st["v_scale"], st["new_v"])):
        if c["kind"] == "bf16":
            val = new.double()
        else:
            top = LEVELS[c["kind"]]
            s = (new.double().abs().max(-1).values / top).float().half().double()
            s[s == 0] = 1.0
            # the quotient is rounded to 32 bits before it is rounded to a code: that is the definition
            val = (new.double() / s[..., None]).float().round().clamp(-top, top).double() * s[..., None]
        old = _row64(c["kind"], codes[page, :, off], None if scale is None else scale[page, :, off])
        old[fresh] = val[pick[fresh]]
        got.append(old)
    return tuple(got)


def _exact_norm(st):
    y, x = st["y"].double(), st["x"].double()
    if st["post"] is not None:
        y = st["post"].double() * y / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    if st["gate"] is not None:
        y = st["gate"].double() * y
    x = st["res"] * x + st["blk"] * y
    return x, st["pre"].double() * x / (x.pow(2).mean(1, keepdim=True) + EPS).sqrt()


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        weights = case["width"] * (2 if case["post"] else 1)
        gate = {"none": 0, "channel": case["width"], "token": n}[case["gate"]]
        return {"bytes": 2 * (4 * n + weights + gate), "flops": n * (12 if case["post"] else 8)}
    lens = lengths(case)
    row = 2 * case["kv_heads"] * (case["dim"] * BITS[case["kind"]] / 8 + (0 if case["kind"] == "bf16" else 2))
    plain = 2 * case["kv_heads"] * case["dim"] * 2
    if case["op"] == "attn":
        pages = sum(-(-n // case["page"]) for n in lens)
        qo = 2 * 2 * case["batch"] * case["heads"] * case["dim"]
        return {"bytes": sum(lens) * row + qo + 4 * (pages + case["batch"]),
                "flops": 4 * sum(lens) * case["heads"] * case["dim"]}
    new = sum(min(case["new"], n) for n in lens)
    # what is read back of the new tokens is still at hand, the rest is read from the cache
    return {"bytes": new * (plain + row + 4) + (sum(lens) - new) * row + sum(lens) * (plain + 4),
            "flops": (6 * new + sum(lens)) * 2 * case["kv_heads"] * case["dim"]}
