"""One token step of a decoder stack on the library's calls: the W4 (+EC)
linears, the key-value cache, the attention over it and the norms between.

Per layer, for one new token of each of n_seqs sequences (all on the device):

    q, k, v = Wq h, Wk h, Wv h
    the cache takes k and v at the token's slots
    x, h = block_norm(x, Wo attention(q, cache))
    x, h = block_norm(x, Wd (silu(Wg h) * Wu h))

with h = norm(x) before the first layer.  Nothing is allocated on the host or
synchronised, so a step can be captured in a CUDA graph: the lengths, slots and
page table are read from the device when it runs.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import spear as S


@dataclass
class StepState:
    """What a decoder keeps between steps: a cache per layer, over one page
    table, the sequences' lengths and the new tokens' slots, and workspaces."""

    caches: list[S.KVCache]
    page_table: torch.Tensor   # n_seqs x max_pages int32
    seq_lens: torch.Tensor     # n_seqs int32, the new token counted
    slots: torch.Tensor        # n_seqs int32, of the new token
    ws: torch.Tensor           # of the linears
    attn_ws: torch.Tensor      # of the attention and the cache calls


def make_state(layers: list, n_seqs: int, max_tokens: int, kind: int = S.KV_INT8, page_size: int = 16,
               head_dim: int = 128) -> StepState:
    """Empty caches for n_seqs sequences of at most max_tokens tokens.  layers: rows
    of seven prepared layers (q, k, v, o, gate, up, down)."""
    dev = layers[0][0].w_packed.device
    n_q, n_kv = layers[0][0].N // head_dim, layers[0][1].N // head_dim
    per_seq = -(-max_tokens // page_size)
    caches = [S.make_kv_cache(kind, n_seqs * per_seq, page_size, n_kv, head_dim, dev) for _ in layers]
    table = torch.arange(n_seqs * per_seq, dtype=torch.int32, device=dev).view(n_seqs, per_seq)
    zeros = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
    ws_bytes = max(S.workspace_bytes(lay, n_seqs) for row in layers for lay in row)
    return StepState(caches, table, zeros, zeros.clone(), torch.zeros(ws_bytes, dtype=torch.uint8, device=dev),
                     S.make_attn_workspace(caches[0], n_q))


def advance(state: StepState) -> None:
    """Count one new token for every sequence and find its slot.  A token past the
    sequence's pages has none: it is not cached, and the attention, whose length
    is then past the table, reports it (`status`)."""
    P, pages = state.caches[0].page_size, state.page_table.shape[1]
    at = state.seq_lens
    page = state.page_table.gather(1, (at // P).clamp(0, pages - 1).long().unsqueeze(1)).squeeze(1)
    state.slots.copy_(torch.where((at >= 0) & (at < pages * P), page * P + at % P, -1))
    state.seq_lens.add_(1)


def step(layers: list, x: torch.Tensor, state: StepState, *, norms: list | None = None, rotate=None,
         eps: float = 1e-6) -> torch.Tensor:
    """x (n_seqs x width bf16) through the layers, for the tokens that the last
    `advance` counted.  norms: per layer the weights (before attention, before
    the MLP), ones if None; rotate: q, k -> q, k, the positional encoding, if any.
    Returns the last layer's x."""
    w = norms if norms is not None else [(None, None)] * len(layers)
    _, h = S.block_norm(x, pre_weight=w[0][0], eps=eps)
    for i, (Lq, Lk, Lv, Lo, Lg, Lu, Ld) in enumerate(layers):
        q, k, v = (S.forward(lay, h, state.ws) for lay in (Lq, Lk, Lv))
        if rotate is not None:
            q, k = rotate(q, k)
        S.kv_write(state.caches[i], k, v, state.slots, state.attn_ws)
        a = S.attn_decode(q, state.caches[i], state.page_table, state.seq_lens, state.attn_ws)
        x, h = S.block_norm(x, S.forward(Lo, a, state.ws), pre_weight=w[i][1], eps=eps)
        gate, up = S.forward(Lg, h, state.ws).float(), S.forward(Lu, h, state.ws).float()
        y = S.forward(Ld, (gate * torch.sigmoid(gate) * up).to(torch.bfloat16), state.ws)
        last = i + 1 == len(layers)
        x, h = S.block_norm(x, y, pre_weight=None if last else w[i + 1][0], norm=not last, eps=eps)
    return x


def status(state: StepState) -> int:
    """An error that the device reported in the steps since the last look, 0 if none:
    the linears' where there is one, else the cache's and the attention's.  Clears
    both workspaces' words (synchronises)."""
    of_linears, of_attention = S.read_status(state.ws), S.read_status(state.attn_ws)
    return of_linears or of_attention
