"""Paged cache: append, read back and attention on the GPU, against the
definitions in 64 bits (paged_util)."""
import math

import pytest
import torch

import paged_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from llama_decoder_forward_gb300 import smol
    return smol


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def starts(news):
    s = [0]
    for n in news:
        s.append(s[-1] + n)
    return s


def fill(S, cache, lens, seed=1, spread=0):
    """Appends random keys and values at positions 0 .. lens[b] - 1, the values' rows times 2^-spread .. 2^spread."""
    B, T = len(lens), max(max(lens), 1)
    shape = (cache.n_layers, B, T, cache.n_kv_heads, cache.head_dim)
    g = torch.Generator("cuda").manual_seed(seed + 2)
    by = torch.exp2(torch.randint(-spread, spread + 1, (*shape[:-1], 1), generator=g, device="cuda").float())
    S.paged_append(cache, S.Chunk(B, T, i32([0] * B), n_new=i32(lens)), randn(*shape, seed=seed),
                   (randn(*shape, seed=seed + 1).float() * by).to(torch.bfloat16))


# ---------------------------------------------------------------- append and read
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd,KV,page,L", [(64, 3, 16, 2), (128, 4, 64, 1), (64, 1, 256, 3), (128, 5, 32, 2)])
def test_append_then_read(S, kind, hd, KV, page, L):
    lens, news, cols = [0, 5, 16, 300, 31], [7, 1, 0, 40, 33], -(-340 // page)
    cache = U.make_cache(S, kind, L, KV, hd, page, 5, cols)
    before = [t.clone().view(torch.uint8) if t is not None and t.dtype != torch.float32 else t for t in cache.tensors]
    rows = starts(news)[-1] + 3                       # three rows behind the last sequence
    k, v = randn(L, rows, KV, hd, seed=3), randn(L, rows, KV, hd, seed=4, scale=30.0)
    S.paged_append(cache, S.Chunk(5, 40, i32(lens), row_start=i32(starts(news))), k, v)
    written = torch.zeros(cache.tensors[0].shape[1:4], dtype=torch.bool, device="cuda")
    for b in range(5):
        at = torch.arange(lens[b], lens[b] + news[b], device="cuda")
        written[cache.tensors[2][b][at // page].long(), :, at % page] = True
        for which, new in (("k", k), ("v", v)):
            want = new[:, starts(news)[b]:starts(news)[b] + news[b]].transpose(1, 2)       # [L, KV, n, hd]
            for layer in range(L):
                got = U.values(cache, which, layer, b, lens[b] + news[b])[:, lens[b]:]
                if kind == "e4m3":
                    codes, scale = U.quantised(want[layer])
                    assert torch.equal(got, codes.double() * scale.double()[..., None])
                    # half a step of e4m3 (2^-4 of the value; below 2^-6 of a unit 2^-10 units), and the
                    # scale's own rounding
                    unit = scale.double()[..., None]
                    bound = torch.maximum(want[layer].double().abs() * 2.0 ** -4, unit * 2.0 ** -10) + unit * 448 * 2.0 ** -23
                    assert ((got - want[layer].double()).abs() <= bound).all()
                else:
                    assert torch.equal(got, want[layer].double())
    for pages, old in zip(cache.tensors[:2], before[:2]):       # nothing else changed
        now = pages.view(torch.uint8).view(*old.shape)
        assert torch.equal(now[:, ~written], old[:, ~written])
    # back into the dense cache of the decode step; slots behind the count stay as they were
    dense = [torch.full((L, 5, KV, 41, hd), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    chunk = S.Chunk(5, 41, i32(lens), n_new=i32(news))
    S.paged_read(cache, chunk, dense[0].transpose(2, 3), dense[1].transpose(2, 3))
    for which, d in zip("kv", dense):
        for b in range(5):
            for layer in range(L):
                want = U.values(cache, which, layer, b, lens[b] + news[b])[:, lens[b]:].float().to(torch.bfloat16)
                assert torch.equal(d[layer, b, :, :news[b]], want)
            assert bool((d[:, b, :, news[b]:] == -7.0).all())


def test_quantised_zero_infinite_and_tiny_rows(S):
    cache = U.make_cache(S, "e4m3", 1, 2, 64, 16, 1, 2)
    k = randn(1, 1, 6, 2, 64, seed=5)
    k[0, 0, 0] = 0
    k[0, 0, 1, 0, 17] = math.inf
    k[0, 0, 2, 1, 63] = math.nan
    k[0, 0, 3] *= 1e-37
    k[0, 0, 4] *= 2.0 ** 100
    k[0, 0, 5, 0] = 0
    k[0, 0, 5, 0, 0] = -3.0
    v = -k
    S.paged_append(cache, S.Chunk(1, 6, i32([9])), k, v)
    out = torch.zeros_like(k)
    vout = torch.zeros_like(k)
    S.paged_read(cache, S.Chunk(1, 6, i32([9])), out, vout)
    got = out[0, 0]
    assert bool((got[0] == 0).all()) and bool((vout[0, 0, 0] == 0).all())
    assert bool(got[1, 0].isnan().all()) and bool(got[2, 1].isnan().all())
    assert bool(got[1, 1].isfinite().all()) and bool(got[2, 0].isfinite().all())
    assert got[5, 0, 0] == -3.0 and bool((got[5, 0, 1:] == 0).all())
    for t in (3, 4):
        unit = k[0, 0, t].double().abs().amax(-1, keepdim=True) / 448
        bound = torch.maximum(k[0, 0, t].double().abs() * 2.0 ** -4, unit * 2.0 ** -10) * (1 + 2.0 ** -7) + unit * 448 * 2.0 ** -8
        assert ((got[t].double() - k[0, 0, t].double()).abs() <= bound).all()


def test_rows_out_of_range_are_not_written(S):
    cache = U.make_cache(S, "bf16", 1, 1, 64, 16, 4, 2)
    cache.tensors[2][1, 1] = cache.n_pages            # no such page
    cache.tensors[2][2, 0] = -1
    before = cache.tensors[0].clone()
    x = randn(1, 4, 3, 1, 64, seed=6)
    # sequence 0 runs over its last page, 1 and 2 name pages that are not there, 3 starts before 0
    chunk = S.Chunk(4, 3, i32([31, 15, 0, -5]))
    S.paged_append(cache, chunk, x, x)
    now = cache.tensors[0]
    changed = (now.view(torch.int16) != before.view(torch.int16)).any(-1).nonzero().tolist()
    t = cache.tensors[2].tolist()
    want = sorted([[0, t[0][1], 0, 15], [0, t[1][0], 0, 15]] + [[0, t[3][0], 0, i] for i in range(3)])
    assert sorted(changed) == want
    out = torch.full_like(x, -7.0)
    S.paged_read(cache, chunk, out, out.clone())
    assert bool((out[0, 0, 1:] == -7).all()) and bool((out[0, 1, 1:] == -7).all()) and bool((out[0, 2] == -7).all())
    assert torch.equal(out[0, 0, 0], x[0, 0, 0])


# ---------------------------------------------------------------- attention
def check_attention(S, kind, H, KV, hd, page, lens, news, window=0, packed=True, scale=None, qscale=2.0, T=None, L=1, layer=0,
                    spread=0):
    B, T = len(lens), T or max(max(news), 1)
    cols = -(-(max(a + n for a, n in zip(lens, news)) + 1) // page)
    cache = U.make_cache(S, kind, L, KV, hd, page, B, cols, seed=len(lens) + H)
    fill(S, cache, [a + n for a, n in zip(lens, news)], spread=spread)
    if packed:
        rs = starts(news)
        rows = rs[-1] + 2
        q = randn(rows, H, hd, seed=9, scale=qscale)
        chunk = S.Chunk(B, T, i32(lens), row_start=i32(rs))
        take = lambda t, b: t[rs[b]:rs[b] + news[b]]
    else:
        q = randn(B, H, T, hd, seed=9, scale=qscale).transpose(1, 2)      # as the projection lays heads out
        chunk = S.Chunk(B, T, i32(lens), n_new=i32(news))
        take = lambda t, b: t[b, :news[b]]
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    ws = S.alloc_paged_workspace(cache, H, B, T)
    S.paged_attention(cache, layer, chunk, q, out, ws, scale=scale or 0.0, window=window)
    assert S.workspace_status(ws) == S.OK
    again = torch.full_like(out, -7.0)
    S.paged_attention(cache, layer, chunk, q, again, ws, scale=scale or 0.0, window=window)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    untouched = torch.ones(out.shape[:-2], dtype=torch.bool, device="cuda")
    for b in range(B):
        take(untouched, b)[...] = False
        if news[b] == 0:
            continue
        k, v = (U.values(cache, x, layer, b, lens[b] + news[b]) for x in "kv")
        ref, mass = U.attention(take(q, b), k, v, lens[b], window, scale or 1 / math.sqrt(hd))
        got = take(out, b).double()
        # half a bf16 step of the output and of each weight (2^-8 relative each), and 2^-12 of the
        # weighted magnitudes for fp32 scores up to some tens and sums over the keys
        bound = ref.abs() * 2.0 ** -8 + mass * (2.0 ** -8 + 2.0 ** -12)
        err = (got - ref).abs()
        assert bool(got.isfinite().all()), f"sequence {b}"
        assert bool((err <= bound).all()), f"sequence {b}: {float((err / bound).max()):.3f} of the bound"
    assert bool((out[untouched] == -7.0).all())


HEADS = [(9, 3, 64), (12, 4, 64), (16, 4, 128), (8, 1, 128), (5, 5, 64), (7, 1, 64), (12, 2, 128), (10, 2, 64)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KV,hd", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(S, kind, H, KV, hd, page):
    # empty caches, one key, borders of pages and tiles, long ones
    lens = [0, 1, 15, 16, 17, 63, 64, 127, 128, 129, 255, 256, 500, 1000, 2049]
    check_attention(S, kind, H, KV, hd, page, lens, [1] * len(lens), packed=False)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KV,hd", HEADS)
@pytest.mark.parametrize("T", [2, 5, 8, 17])
def test_drafted_rows(S, kind, H, KV, hd, T):
    lens = [0, 3, 60, 200, 777, 1500]
    check_attention(S, kind, H, KV, hd, 32, lens, [T] * len(lens), packed=False)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KV,hd", [(9, 3, 64), (16, 4, 128), (7, 1, 64), (8, 1, 128), (3, 3, 128)])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_ragged_chunks(S, kind, H, KV, hd, window):
    check_attention(S, kind, H, KV, hd, 16, [0, 100, 513, 0, 40, 1023], [300, 1, 129, 0, 64, 257], window=window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KV,hd", [(9, 3, 64), (16, 4, 128)])
def test_padded_batch(S, kind, H, KV, hd):
    check_attention(S, kind, H, KV, hd, 128, [5, 0, 700], [90, 0, 33], packed=False, T=100)


@pytest.mark.parametrize("kind,hd", [("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("window", [1, 3, 64, 65, 129, 5000])
def test_windows(S, kind, hd, window):
    check_attention(S, kind, 6, 2, hd, 16, [0, 10, 130, 1000], [3, 3, 3, 3], window=window)
    check_attention(S, kind, 6, 2, hd, 16, [0, 130, 1000], [200, 150, 270], window=window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_long_cache_and_long_chunk(S, kind):
    check_attention(S, kind, 4, 1, 64, 256, [40000, 3], [1, 1], packed=False)
    check_attention(S, kind, 4, 1, 128, 64, [20000], [600])


def test_many_sequences(S):
    n = 700
    lens, news = [(37 * i) % 90 for i in range(n)], [(i * 7) % 4 for i in range(n)]
    check_attention(S, "bf16", 6, 3, 64, 16, lens, news)


def test_scale_and_large_scores(S):
    check_attention(S, "bf16", 4, 2, 64, 16, [300], [70], scale=0.5)
    check_attention(S, "bf16", 4, 2, 64, 16, [300, 20], [1, 1], scale=0.5)
    # scores of some hundreds: one key takes all the weight
    check_attention(S, "bf16", 4, 2, 64, 16, [300, 7], [5, 5], qscale=0.25, scale=8.0)


def test_layers_of_one_pool(S):
    for layer in (0, 2):
        check_attention(S, "e4m3", 8, 2, 64, 32, [50, 333], [4, 80], L=3, layer=layer)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KV,hd,T", [(8, 1, 64, 1), (8, 1, 64, 3), (8, 1, 64, 4), (8, 1, 64, 6), (7, 1, 64, 7), (6, 1, 64, 8),
                                       (8, 1, 128, 1), (8, 1, 128, 2), (8, 1, 128, 3), (8, 1, 128, 4), (5, 1, 128, 9),
                                       (1, 1, 128, 9), (1, 1, 64, 33), (3, 1, 128, 16), (7, 1, 128, 18)])
def test_rows_next_to_the_kernels_borders(S, kind, H, KV, hd, T):
    check_attention(S, kind, H, KV, hd, 16, [0, 31, 500, 1200, 2], [T, T, max(T - 2, 0), T, 1], packed=False)


def test_strides_of_axes_of_one_entry_say_nothing(S):
    import ctypes
    cache = U.make_cache(S, "bf16", 1, 1, 64, 16, 1, 4)
    fill(S, cache, [40])
    q, out, ws = randn(1, 1, 1, 64, seed=8), torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda"), S.alloc_paged_workspace(cache, 1, 1, 64)
    chunk = S.Chunk(1, 1, i32([39]))
    S.paged_attention(cache, 0, chunk, q, out, ws)
    bare = torch.zeros_like(out)
    rows = [ctypes.byref(S._Rows(t.data_ptr(), 0, 0, 0, 0)) for t in (q, bare)]
    S._check(S._lib.smol_paged_attention(cache.ref, 0, chunk.ref(1), 1, *rows, 0.0, 0, ws.data_ptr(), ws.numel(), S._stream()), "attention")
    assert S.workspace_status(ws) == S.OK
    assert torch.equal(out, bare)
    # the many-rows kernel: one head, one sequence
    q, out = randn(1, 40, 1, 64, seed=9), torch.zeros(1, 40, 1, 64, dtype=torch.bfloat16, device="cuda")
    chunk = S.Chunk(1, 40, i32([0]))
    S.paged_attention(cache, 0, chunk, q, out, ws)
    bare = torch.zeros_like(out)
    rows = [ctypes.byref(S._Rows(t.data_ptr(), 0, 0, 64, 0)) for t in (q, bare)]
    S._check(S._lib.smol_paged_attention(cache.ref, 0, chunk.ref(1), 1, *rows, 0.0, 0, ws.data_ptr(), ws.numel(), S._stream()), "attention")
    assert torch.equal(out, bare)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KV,hd", [(9, 3, 64), (16, 4, 128)])
def test_values_of_very_different_size(S, kind, H, KV, hd):
    # the first row sees neither the last positions nor, with a window, the first ones
    for T in (1, 4, 5, 9, 100):
        check_attention(S, kind, H, KV, hd, 16, [0, 40, 700], [T, T, T], packed=False, spread=40, window=0 if T % 2 else 50)
    # peaked: the large values have weights of next to nothing
    check_attention(S, kind, H, KV, hd, 16, [300, 90], [3, 70], spread=30, qscale=8.0)
