"""What the header promises of the paged operators beyond single calls: one workspace
for calls of every size, rows out of range that leave memory as it was."""
import math

import pytest
import torch

import paged_util as U
from parity_util import LOGITS_COS_MIN, LOGITS_MAX_ABS, cosine, max_abs, np32
from test_gpu_paged_model import S, case, i32, randn, small  # noqa: F401 (S is a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- one workspace
@pytest.mark.parametrize("kind,hd128", [("bf16", False), ("e4m3", True)])
def test_one_workspace_serves_prompts_drafts_and_single_tokens(S, kind, hd128):
    """Zeroed once, of the largest call's size: in the larger calls its bytes hold activations where a smaller
    call's own layout would end.  The caches are long enough that units are shared by several CTAs."""
    lengths = [0, 1200, 64, 5, 2500]
    wl, _, _, cfg, packed, cache, ids = case(S, 71, lengths, 70, kind=kind, hd128=hd128)
    ws = S.prefill_paged_workspace(cfg, cache, 5, 70)

    def forward(B, T, w):
        logits = torch.full((B, T, wl.vocab), math.nan, dtype=torch.bfloat16, device="cuda")
        S.prefill_paged(cfg, packed, ids[:B, :T].contiguous().cuda(), cache, i32(lengths[:B]), logits, w)
        assert S.workspace_status(w) == S.OK
        return np32(logits)

    for B, T in [(5, 70), (5, 1), (2, 5), (5, 5), (2, 1), (2, 70), (5, 1), (5, 70), (5, 5)]:
        got, want = forward(B, T, ws), forward(B, T, S.prefill_paged_workspace(cfg, cache, B, T))
        # two runs of one call (the order of the sums of squares may differ): each within the bar of the definition
        assert cosine(got, want) >= LOGITS_COS_MIN and max_abs(got, want) <= 2 * LOGITS_MAX_ABS, (B, T)


# ---------------------------------------------------------------- rows out of range
def bits(cache):
    return [None if t is None else t.clone().view(torch.uint8) for t in cache.tensors]


def unchanged(cache, before, rows):
    """Nothing in the pools but the rows [(page, slot)] of every layer and kv head has changed."""
    for now, old in zip(bits(cache), before):
        if now is None or now.dim() < 4:
            continue
        now, old = (t.flatten(4) if t.dim() > 4 else t.view(*t.shape[:3], cache.page_size, -1) for t in (now, old))
        differs = (now != old).flatten(4).any(-1).any(2).any(0)                # [page, slot]
        for page, slot in rows:
            differs[page, slot] = False
        if bool(differs.any()):
            return False
    return True


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 7])
def test_a_negative_position_moves_no_rows(S, kind, T):
    """-5 + 6 would be a position again; the whole sequence is left out."""
    cache = small(S, kind, T, [20, 20, 20])
    before = bits(cache)
    k, v = randn(1, 3, T, 2, 64, seed=31), randn(1, 3, T, 2, 64, seed=32)
    chunk = S.Chunk(3, T, i32([-5, 20, -2 ** 31]))
    S.paged_append(cache, chunk, k, v)
    at = [20 + t for t in range(T)]
    ids = cache.tensors[2][1].tolist()
    assert unchanged(cache, before, [(ids[x // 16], x % 16) for x in at])
    for which, new in (("k", k), ("v", v)):
        want = new[0, 1].transpose(0, 1)                                         # [KV, T, hd]
        if kind == "e4m3":
            codes, scale = U.quantised(want)
            want = codes.double() * scale.double()[..., None]
        assert torch.equal(U.values(cache, which, 0, 1, 20 + T)[:, 20:], want.double())
    out = [torch.full((1, 3, T, 2, 64), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    S.paged_read(cache, chunk, *out)
    for o in out:
        assert bool((o[0, [0, 2]] == -7.0).all()) and not bool((o[0, 1] == -7.0).any())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_negative_start_moves_no_rows(S, kind):
    cache = small(S, kind, 8, [20, 20, 20])
    before = bits(cache)
    k, v = randn(1, 12, 2, 64, seed=33), randn(1, 12, 2, 64, seed=34)
    chunk = S.Chunk(3, 8, i32([4, 20, 9]), row_start=i32([-3, 4, 8, 12]))
    S.paged_append(cache, chunk, k, v)
    table = cache.tensors[2].tolist()
    rows = [(table[b][x // 16], x % 16) for b, at in ((1, 20), (2, 9)) for x in range(at, at + 4)]
    assert unchanged(cache, before, rows)
    out = [torch.full((1, 12, 2, 64), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    S.paged_read(cache, chunk, *out)
    for o, new in zip(out, (k, v)):
        assert bool((o[0, :4] == -7.0).all())
        if kind == "bf16":
            assert torch.equal(o[0, 4:], new[0, 4:])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_model_leaves_the_pages_of_a_negative_position(S, kind):
    lengths = [4, 20]
    wl, _, _, cfg, packed, cache, ids = case(S, 12, lengths, 3, kind=kind)
    before = bits(cache)
    logits = torch.zeros(2, 3, wl.vocab, dtype=torch.bfloat16, device="cuda")
    ws = S.prefill_paged_workspace(cfg, cache, 2, 3)
    S.prefill_paged(cfg, packed, ids.cuda(), cache, i32([-1, 20]), logits, ws)
    assert S.workspace_status(ws) == S.ERR_INPUT
    table = cache.tensors[2].tolist()
    assert unchanged(cache, before, [(table[1][x // 16], x % 16) for x in range(20, 23)])


# ---------------------------------------------------------------- waits that give up
def gives_up(S, kind, hd, T, lens):
    """A call under a limit of a nanosecond, three times: its statuses.  What did not give up is right, and the
    workspace serves the call behind each."""
    cache = small(S, kind, T, [n + T for n in lens], hd=hd)
    q = randn(len(lens), T, 6, hd, seed=4, scale=2.0)
    chunk, ws = S.Chunk(len(lens), T, i32(lens)), S.alloc_paged_workspace(cache, 6, len(lens), T)
    want, out = torch.empty_like(q), torch.empty_like(q)
    S.paged_attention(cache, 0, chunk, q, want, ws)
    assert S.workspace_status(ws) == S.OK
    flush, reports = torch.empty(256 << 20, dtype=torch.uint8, device="cuda"), []
    for _ in range(3):
        flush.fill_(1)                                # the pages come from memory, not from L2
        try:
            S.set_wait_limit_ns(1)
            S.paged_attention(cache, 0, chunk, q, out, ws)
            reports.append(S.workspace_status(ws))
        finally:
            S.set_wait_limit_ns(0)
        assert reports[-1] == S.ERR_TIMEOUT or (reports[-1] == S.OK and torch.equal(out, want))
        S.paged_attention(cache, 0, chunk, q, out, ws)
        assert S.workspace_status(ws) == S.OK and torch.equal(out, want)
    return reports


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T", [40, 100])
@pytest.mark.parametrize("lens", [[900, 6000, 31] + [5000] * 13, [40, 0, 200]])
def test_many_rows_keep_a_short_wait_limit(S, kind, hd, T, lens):
    """Pieces of many key tiles, and of one or two, whose copies are all asked for when the first wait gives up."""
    assert gives_up(S, kind, hd, T, lens) == 3 * [S.ERR_TIMEOUT]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
def test_few_rows_keep_a_short_wait_limit(S, kind, hd):
    """The first keys of 150 MB, which all the SMs ask for at once.  A kernel whose steps take longer than its copies
    (32 rows over codes) never waits, and a small call's copies may be there in time: those are right instead."""
    reports = []
    for T in (1, 3, 6, 8):
        reports += gives_up(S, kind, hd, T, [6000] * (48 if kind == "bf16" else 96))
        gives_up(S, kind, hd, T, [40, 0, 200])
    assert reports.count(S.ERR_TIMEOUT) >= 3, reports


def test_the_model_over_pages_reports_a_wait_that_gave_up(S):
    lengths = [3, 900, 40]
    wl, _, _, cfg, packed, cache, ids = case(S, 13, lengths, 30)
    ws = S.prefill_paged_workspace(cfg, cache, 3, 30)
    for T in (30, 1):
        logits, want = (torch.zeros(3, T, wl.vocab, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        call = lambda to: S.prefill_paged(cfg, packed, ids[:, :T].contiguous().cuda(), cache, i32(lengths), to, ws)
        call(want)
        assert S.workspace_status(ws) == S.OK
        try:
            S.set_wait_limit_ns(1)
            call(logits)
            assert S.workspace_status(ws) == S.ERR_TIMEOUT
        finally:
            S.set_wait_limit_ns(0)
        call(logits)
        assert S.workspace_status(ws) == S.OK
        assert cosine(np32(logits), np32(want)) >= LOGITS_COS_MIN and max_abs(np32(logits), np32(want)) <= 2 * LOGITS_MAX_ABS


# ---------------------------------------------------------------- the launch timer
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_timer_files_chunks_of_prompts_under_prefill_attention(S, kind):
    cache = small(S, kind, 100, [300, 40])
    ws = S.alloc_paged_workspace(cache, 6, 2, 100)
    for T, want in ((1, [S.K_DEC_ATTN]), (4, [S.K_DEC_ATTN]), (100, [S.K_ATTN, S.K_ATTN])):
        q = randn(2, T, 6, 64, seed=T)
        S.profile_begin((1 << len(S.KERNEL_KINDS)) - 1, 8)
        S.paged_attention(cache, 0, S.Chunk(2, T, i32([20, 30])), q, torch.empty_like(q), ws)
        assert [k for k, _ in S.profile_end()] == want
