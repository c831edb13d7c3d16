"""Paged caches for the tests, and their operators from the definitions in 64 bits.

The pools are filled with NaN (bf16 pages, scales) before any use, so that a read
of a slot that no call may use shows in the outputs."""
import math

import torch

F8 = torch.float8_e4m3fn


def make_cache(S, kind, L, KV, hd, page, n_seqs, max_pages, seed=0, spare=3):
    """A PagedCache over poisoned pools; every sequence's pages scattered over them."""
    P = n_seqs * max_pages + spare
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(P, generator=g)[:n_seqs * max_pages].to(torch.int32).view(n_seqs, max_pages).cuda()
    shape = (L, P, KV, page, hd)
    if kind == "bf16":
        k, v = (torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return S.PagedCache(k, v, table)
    k, v = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
    ks, vs = (torch.full(shape[:-1], math.nan, device="cuda") for _ in range(2))
    return S.PagedCache(k, v, table, ks, vs)


def values(cache, which, layer, b, n):
    """Positions 0 .. n - 1 of sequence b as the pages hold them: [KV, n, hd] in 64 bits."""
    pages, scale = (cache.tensors[0], cache.tensors[3]) if which == "k" else (cache.tensors[1], cache.tensors[4])
    ids = cache.tensors[2][b].long()
    raw = pages[layer].view(torch.uint8)[ids].view(F8) if cache.e4m3 else pages[layer][ids]
    x = raw.double()                                                    # [pages, KV, page, hd]
    if cache.e4m3:
        x = x * scale[layer][ids].double()[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def attention(q, k, v, pos, window, scale):
    """(out, sum_j p_j |v_j|) of one sequence's rows: q [n, H, hd], k and v [KV, pos + n, hd], in 64 bits."""
    n, H, _ = q.shape
    G = H // k.shape[0]
    k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    s = torch.einsum("nhd,hjd->hnj", q.double(), k) * scale
    at = pos + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(k.shape[1], device=q.device)
    hidden = j > at
    if window:
        hidden |= j <= at - window
    # what a row does not see is left out of its sums, whatever it holds
    p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
    seen = (~hidden).any(0)[None, :, None]
    v = torch.where(seen, v, torch.zeros((), dtype=v.dtype, device=v.device))
    return torch.einsum("hnj,hjd->nhd", p, v), torch.einsum("hnj,hjd->nhd", p, v.abs())


def quantised(x):
    """(codes, scales) of rows of bf16: the definition, with the division in 32 bits."""
    x = x.float()
    scale = x.abs().amax(-1) / torch.tensor(448.0, device=x.device)
    codes = (x / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]).to(F8)
    return codes, scale
