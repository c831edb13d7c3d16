"""The model over a paged cache (smol_prefill_paged) against the oracle, and the
paged operators as a serving loop uses them: append, attend, verify, one behind the
other, captured into graphs, on streams, and with inputs out of range."""
import math

import numpy as np
import pytest
import torch

import paged_util as U
from llama_decoder_forward_gb300 import synth
from oracle import oracle as O
from parity_util import LOGITS_COS_MIN, LOGITS_MAX_ABS, cosine, max_abs, np32, oracle_config, oracle_layers, to_device

pytestmark = pytest.mark.gpu

W = synth.WORKLOADS


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from llama_decoder_forward_gb300 import smol
    return smol


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def case(S, seed, lengths, T, kind="bf16", page=16, hd128=False, **kw):
    """A small model, its pages filled from dense caches, and T new tokens."""
    s_max = max(max(lengths), 1)
    wl = W["smollm2_decode_b64_cache4096"].scaled(B=len(lengths), n_layers=2, s_max=s_max, vocab=512, **kw)
    if hd128:
        wl = wl.scaled(hidden=512, n_heads=4, n_kv_heads=2, head_dim=128, intermediate=768, w_std=0.0442)
    inp = synth.generate(wl, seed=seed)
    inp.lengths = torch.tensor(lengths, dtype=torch.int32)
    dev = to_device(inp)
    cfg = S.config_of(wl)
    packed = S.prepare_weights(cfg, dev.layers, dev.embed, dev.final_norm)
    cache = U.make_cache(S, kind, wl.n_layers, wl.n_kv_heads, wl.head_dim, page, wl.B, -(-(s_max + T) // page), seed=seed)
    S.paged_append(cache, S.Chunk(wl.B, s_max, i32([0] * wl.B), n_new=dev.lengths), dev.k_cache.transpose(2, 3),
                   dev.v_cache.transpose(2, 3))
    ids = torch.randint(0, wl.vocab, (wl.B, T), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    return wl, inp, dev, cfg, packed, cache, ids


def run(S, wl, cfg, packed, cache, ids, lengths):
    logits = torch.full((wl.B, ids.shape[1], wl.vocab), math.nan, dtype=torch.bfloat16, device="cuda")
    ws = S.prefill_paged_workspace(cfg, cache, wl.B, ids.shape[1])
    S.prefill_paged(cfg, packed, ids.cuda(), cache, i32(lengths), logits, ws)
    assert S.workspace_status(ws) == S.OK
    return logits


@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("kw", [dict(), dict(hd128=True), dict(no_rope_layers=(1, 0), sliding_window=(0, 9))])
def test_prefill_paged_against_the_oracle(S, T, kw):
    lengths = [0, 37, 64, 5, 130]
    wl, inp, dev, cfg, packed, cache, ids = case(S, 60 + T, lengths, T, **kw)
    logits = run(S, wl, cfg, packed, cache, ids, lengths)
    ref, kr, vr = O.prefill_with_cache(oracle_config(wl), oracle_layers(inp), np32(inp.embed), np32(inp.final_norm),
                                       ids.numpy().astype(np.int64), np.asarray(lengths), np32(inp.k_cache), np32(inp.v_cache))
    got = np32(logits).astype(np.float64)
    assert cosine(got, ref) >= LOGITS_COS_MIN and max_abs(got, ref) <= LOGITS_MAX_ABS
    for layer in range(2):
        for b, n in enumerate(lengths):
            for which, want in (("k", kr), ("v", vr)):
                new = U.values(cache, which, layer, b, n + T)[:, n:].cpu().numpy()
                # the bar of the dense calls' new entries: 5e-2 of their RMS, and their own bf16 rounding
                assert np.all(np.abs(new - want[layer, b]) <= 5e-2 * np.sqrt(np.mean(want[layer] ** 2)) + 2.0 ** -8 * np.abs(want[layer, b]))


def test_prefill_paged_quantises_what_it_writes(S):
    lengths = [3, 50]
    got = {}
    for kind in ("bf16", "e4m3"):
        wl, _, _, cfg, packed, cache, ids = case(S, 9, lengths, 6, kind=kind)
        logits = run(S, wl, cfg, packed, cache, ids, lengths)
        assert bool(logits.isfinite().all())
        got[kind] = [[U.values(cache, w, 0, b, n + 6)[:, n:] for b, n in enumerate(lengths)] for w in "kv"]
    # the first block's keys and values do not depend on the cache: the codes are those of the bf16 run's
    for a, b in zip(got["bf16"], got["e4m3"]):
        for x, y in zip(a, b):
            codes, scale = U.quantised(x.to(torch.bfloat16))
            assert torch.equal(codes.double() * scale.double()[..., None], y)


def test_prefill_paged_records_lengths_out_of_range(S):
    lengths = [4, 20]
    wl, _, _, cfg, packed, cache, ids = case(S, 10, lengths, 3)
    logits = torch.zeros(2, 3, wl.vocab, dtype=torch.bfloat16, device="cuda")
    ws = S.prefill_paged_workspace(cfg, cache, 2, 3)
    for bad in ([-1, 20], [4, cache.max_pages * 16 - 2]):
        S.prefill_paged(cfg, packed, ids.cuda(), cache, i32(bad), logits, ws)
        assert S.workspace_status(ws) == S.ERR_INPUT
    S.prefill_paged(cfg, packed, ids.cuda(), cache, i32(lengths), logits, ws)
    assert S.workspace_status(ws) == S.OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_speculative_greedy_follows_the_sequential_one(S, kind):
    """Drafts that are the sequential run's tokens, some of them replaced: what stays and what comes next are
    the sequential run's tokens, wherever its choice was clear."""
    lengths, steps, T = [0, 21, 40], 18, 4
    wl, _, _, cfg, packed, cache, ids = case(S, 31, lengths, steps + T + 2, kind=kind)
    start = ids[:, :1].cuda()
    # one token at a time
    tok, pos = start.clone(), i32(lengths)
    logits = torch.empty(wl.B, 1, wl.vocab, dtype=torch.bfloat16, device="cuda")
    ws = S.prefill_paged_workspace(cfg, cache, wl.B, 1)
    seq, margin = [start[:, 0].clone()], []
    for _ in range(steps + T + 1):
        S.prefill_paged(cfg, packed, tok, cache, pos, logits, ws)
        top = logits[:, 0].float().topk(2).values
        margin.append(top[:, 0] - top[:, 1])
        nxt = torch.empty(wl.B, dtype=torch.int32, device="cuda")
        S.sample(logits[:, 0], nxt, do_sample=False)
        seq.append(nxt.clone())
        tok = nxt[:, None].contiguous()
        pos += 1
    assert S.workspace_status(ws) == S.OK
    seq, margin = torch.stack(seq, 1), torch.stack(margin, 1)               # [B, n]
    # T drafts at a time over the same pages (the sequential run's entries behind pos are overwritten)
    g = torch.Generator("cuda").manual_seed(5)
    pos, done = i32(lengths), torch.zeros(wl.B, dtype=torch.long, device="cuda")
    logits = torch.empty(wl.B, T + 1, wl.vocab, dtype=torch.bfloat16, device="cuda")
    ws, vws = S.prefill_paged_workspace(cfg, cache, wl.B, T + 1), S.alloc_verify_workspace(wl.B, T)
    acc, nxt = (torch.empty(wl.B, dtype=torch.int32, device="cuda") for _ in range(2))
    clear = torch.ones(wl.B, dtype=torch.bool, device="cuda")
    while bool((done < steps).any()):
        at = (done[:, None] + torch.arange(T + 1, device="cuda")).clamp_max(seq.shape[1] - 1)
        chunk = seq.gather(1, at).to(torch.int32)
        wrong = torch.rand(wl.B, T, generator=g, device="cuda") < 0.25
        chunk[:, 1:] = torch.where(wrong, (chunk[:, 1:] + 1) % wl.vocab, chunk[:, 1:])
        S.prefill_paged(cfg, packed, chunk.contiguous(), cache, pos, logits, ws)
        S.verify_drafts(logits, chunk[:, 1:].contiguous(), acc, nxt, vws, do_sample=False)
        for b in range(wl.B):
            n, i = int(acc[b]), int(done[b])
            # two runs' logits differ by two bars at most: choices nearer than that may part
            clear[b] &= bool((margin[b, i:i + n + 1] > 4 * LOGITS_MAX_ABS).all()) if kind == "bf16" else False
            first_wrong = next((j for j in range(T) if wrong[b, j]), T)
            if clear[b]:
                assert n == first_wrong and int(nxt[b]) == int(seq[b, min(i + n + 1, seq.shape[1] - 1)])
            assert n <= T and int(nxt[b]) == int(logits[b, n].float().argmax())
            if not clear[b] or i + n + 1 >= steps:
                done[b] = steps                                             # parted, or finished
            else:
                done[b] += n + 1
        pos += torch.where(done < steps, acc + 1, torch.zeros_like(acc))
    assert S.workspace_status(ws) == S.OK and S.workspace_status(vws) == S.OK


# ---------------------------------------------------------------- the operators as a program uses them
def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def small(S, kind, T, lens, H=6, KV=2, hd=64, page=16, seed=0):
    cache = U.make_cache(S, kind, 1, KV, hd, page, len(lens), -(-(max(lens) + 2 * T) // page), seed=seed)
    n = max(max(lens), 1)
    S.paged_append(cache, S.Chunk(len(lens), n, i32([0] * len(lens)), n_new=i32(lens)), randn(1, len(lens), n, KV, hd, seed=seed + 1),
                   randn(1, len(lens), n, KV, hd, seed=seed + 2))
    return cache


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 4, 30])
def test_append_and_attend_in_graphs_that_share_a_workspace(S, kind, T):
    lens = [7, 200, 333]
    B, H, KV, hd = 3, 6, 2, 64
    cache = small(S, kind, T, lens)
    pos = i32(lens)
    chunk = S.Chunk(B, T, pos)
    ws = S.alloc_paged_workspace(cache, H, B, T)
    bufs = [[randn(1, B, T, KV, hd, seed=s), randn(1, B, T, KV, hd, seed=s + 1), randn(B, T, H, hd, seed=s + 2, scale=2.0)] for s in (50, 60)]
    outs = [torch.empty(B, T, H, hd, dtype=torch.bfloat16, device="cuda") for _ in bufs]

    def step(i):
        k, v, q = bufs[i]
        S.paged_append(cache, chunk, k, v)
        S.paged_attention(cache, 0, chunk, q, outs[i], ws)

    want = []
    for i in range(2):
        step(i)
        want.append(outs[i].clone())
    graphs = []
    side = torch.cuda.Stream()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(i)
        graphs.append(g)
    for o in outs:
        o.zero_()
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
    # new contents of the same buffers, replayed: what an eager call gives
    new = randn(B, T, H, hd, seed=77, scale=2.0)
    bufs[0][2].copy_(new)
    pos.copy_(i32([3, 190, 320]))
    graphs[0].replay()
    torch.cuda.synchronize()
    got = outs[0].clone()
    step(0)
    assert torch.equal(got, outs[0])
    assert S.workspace_status(ws) == S.OK


@pytest.mark.parametrize("T", [1, 40])
def test_calls_at_once_on_two_streams(S, T):
    cases = []
    for seed in (0, 1):
        lens = [50 + 40 * seed, 900]
        cache = small(S, "bf16", T, lens, seed=10 * seed)
        q = randn(2, T, 6, 64, seed=seed, scale=2.0)
        chunk, ws, out = S.Chunk(2, T, i32([n - T for n in lens])), S.alloc_paged_workspace(cache, 6, 2, T), torch.empty_like(q)
        S.paged_attention(cache, 0, chunk, q, out, ws)
        cases.append((cache, chunk, q, ws, out.clone(), out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for cache, chunk, q, ws, want, out, st in cases:
            with torch.cuda.stream(st):
                S.paged_attention(cache, 0, chunk, q, out, ws)
    torch.cuda.synchronize()
    for *_, want, out, st in cases:
        assert torch.equal(want, out)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,window", [(1, 20), (6, 33), (90, 64)])
def test_poison_before_every_window_is_not_used(S, kind, T, window):
    lens = [300, 77]
    cache = small(S, kind, T, [n + T for n in lens])
    q = randn(2, T, 6, 64, seed=4, scale=2.0)
    chunk, ws = S.Chunk(2, T, i32(lens)), S.alloc_paged_workspace(cache, 6, 2, T)
    out, again = torch.empty_like(q), torch.empty_like(q)
    S.paged_attention(cache, 0, chunk, q, out, ws, window=window)
    for b, n in enumerate(lens):
        at = torch.arange(0, max(0, n - window + 1), device="cuda")      # position n's window starts behind these
        page, slot = cache.tensors[2][b][at // 16].long(), at % 16
        for pages in cache.tensors[:2]:
            if kind == "bf16":
                pages[0, page, :, slot] = math.nan
            else:
                pages.view(torch.uint8)[0, page, :, slot] = 0x7f
        if kind == "e4m3":
            for scale in cache.tensors[3:]:
                scale[0, page, :, slot] = math.nan
    S.paged_attention(cache, 0, chunk, q, again, ws, window=window)
    assert torch.equal(out, again) and bool(out.isfinite().all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 5, 50])
def test_bad_tables_and_lengths_are_recorded(S, kind, T):
    lens = [40, 60, 100]
    cache = small(S, kind, T, lens)
    q, ws = randn(3, T, 6, 64, seed=4), S.alloc_paged_workspace(cache, 6, 3, T)
    good, out = torch.empty_like(q), torch.empty_like(q)
    pos = [n - T if n >= T else 0 for n in lens]
    S.paged_attention(cache, 0, S.Chunk(3, T, i32(pos)), q, good, ws)
    assert S.workspace_status(ws) == S.OK
    cap = cache.max_pages * 16
    for bad in ([-7, pos[1], pos[2]], [cap + 5, pos[1], pos[2]], [cap - T + 1, pos[1], pos[2]]):
        S.paged_attention(cache, 0, S.Chunk(3, T, i32(bad)), q, out, ws)
        assert S.workspace_status(ws) == S.ERR_INPUT
        assert torch.equal(out[1:], good[1:])                             # the other sequences' rows
    for page in (-1, cache.n_pages, 2 ** 31 - 1):
        saved = int(cache.tensors[2][0, 0])
        cache.tensors[2][0, 0] = page
        S.paged_attention(cache, 0, S.Chunk(3, T, i32(pos)), q, out, ws)
        assert S.workspace_status(ws) == S.ERR_INPUT
        assert torch.equal(out[1:], good[1:])
        cache.tensors[2][0, 0] = saved
    # more rows than T, and starts that go back or beyond the tensor
    rows = torch.empty(3 * T, 6, 64, dtype=torch.bfloat16, device="cuda").copy_(q.flatten(0, 1))
    for starts in ([0, 2 * T, 2 * T, 3 * T], [0, T, 2 * T, 3 * T + 9], [-2, T, 2 * T, 3 * T], [0, T, T - 1, 3 * T]):
        S.paged_attention(cache, 0, S.Chunk(3, T, i32(pos), row_start=i32(starts)), rows, torch.empty_like(rows), ws)
        assert S.workspace_status(ws) == S.ERR_INPUT


def test_nothing_to_do(S):
    cache = small(S, "bf16", 4, [5, 5])
    ws = S.alloc_paged_workspace(cache, 6, 2, 4)
    q = randn(2, 4, 6, 64)
    out = torch.full_like(q, -7.0)
    S.paged_attention(cache, 0, S.Chunk(2, 4, i32([0, 3]), n_new=i32([0, 0])), q, out, ws)
    assert S.workspace_status(ws) == S.OK and bool((out == -7).all())
    none = torch.empty(0, 6, 64, dtype=torch.bfloat16, device="cuda")
    S.paged_attention(cache, 0, S.Chunk(2, 4, i32([0, 3]), row_start=i32([0, 0, 0])), none, none.clone(), ws)
    kv = torch.empty(1, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    S.paged_append(cache, S.Chunk(2, 4, i32([0, 3]), row_start=i32([0, 0, 0])), kv, kv.clone())


def test_a_workspace_serves_calls_of_every_kind(S):
    """Few rows, many rows, few rows again on one workspace of the largest size: the counters are left at zero."""
    lens = [500, 1200]
    cache = small(S, "bf16", 64, lens)
    ws = S.alloc_paged_workspace(cache, 6, 2, 64)
    want = {}
    for turn in range(3):
        for T in (1, 9, 64):
            q = randn(2, T, 6, 64, seed=T, scale=2.0)
            out = torch.empty_like(q)
            S.paged_attention(cache, 0, S.Chunk(2, T, i32([n - T for n in lens])), q, out, ws)
            assert torch.equal(out, want.setdefault(T, out))
    assert S.workspace_status(ws) == S.OK


def test_binding_refuses(S):
    cache = small(S, "bf16", 4, [5, 9])
    ws, q = S.alloc_paged_workspace(cache, 6, 2, 4), randn(2, 4, 6, 64)
    chunk = S.Chunk(2, 4, i32([0, 0]))
    for bad in (q.float(), q[:, :3], q[..., :32], q.transpose(2, 3).contiguous().transpose(2, 3), q.cpu()):
        with pytest.raises(ValueError):
            S.paged_attention(cache, 0, chunk, bad, torch.empty_like(q), ws)
    with pytest.raises(S.SmolError):
        S.paged_attention(cache, 0, chunk, q, q[:, :, :1].expand(2, 4, 6, 64), ws)      # rows on one another
    with pytest.raises(S.SmolError):
        S.paged_attention(cache, 3, chunk, q, torch.empty_like(q), ws)
    with pytest.raises(S.SmolError):
        S.paged_attention(cache, 0, chunk, q, torch.empty_like(q), ws[:2048])
    with pytest.raises(ValueError):
        S.paged_attention(cache, 0, S.Chunk(3, 4, i32([0, 0, 0])), randn(3, 4, 6, 64), randn(3, 4, 6, 64), ws)
    with pytest.raises(ValueError):
        S.Chunk(2, 4, i32([0, 0]), row_start=i32([0, 1, 2]), n_new=i32([1, 1]))
    with pytest.raises(ValueError):
        S.PagedCache(cache.tensors[0], cache.tensors[1], cache.tensors[2], torch.zeros(3, device="cuda"), None)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T", [1, 9, 20, 100])
def test_a_wait_that_gives_up_is_reported(S, kind, hd, T):
    """With a wait limit below the kernels' own latencies they give up, say so and leave the device and the
    workspace usable."""
    lens = [900, 6000, 31] + [5000] * 13
    cache = small(S, kind, T, [n + T for n in lens], H=6, KV=2, hd=hd)
    q = randn(len(lens), T, 6, hd, seed=4, scale=2.0)
    chunk, ws = S.Chunk(len(lens), T, i32(lens)), S.alloc_paged_workspace(cache, 6, len(lens), T)
    want, out = torch.empty_like(q), torch.empty_like(q)
    S.paged_attention(cache, 0, chunk, q, want, ws)
    assert S.workspace_status(ws) == S.OK
    try:
        S.set_wait_limit_ns(1)
        S.paged_attention(cache, 0, chunk, q, out, ws)
        status = S.workspace_status(ws)
        # a wait looks several times before it looks at the clock: what comes within that is no failure
        assert status == S.ERR_TIMEOUT or (status == S.OK and torch.equal(out, want))
    finally:
        S.set_wait_limit_ns(0)
    S.paged_attention(cache, 0, chunk, q, out, ws)
    assert S.workspace_status(ws) == S.OK and torch.equal(out, want)
    print(f"T={T}: status {status}")
