"""Verification of drafted tokens on the GPU against the definition in 64 bits
(numpy, one sequence after the other)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from llama_decoder_forward_gb300 import smol
    return smol


def distribution(logits, temperature, top_k, top_p):
    """The target's probabilities of one row, in 64 bits."""
    z = logits.astype(np.float64) / float(np.float32(temperature))
    keep = z > -np.inf
    if 0 < top_k < z.size:
        keep &= z >= np.sort(z)[-top_k]
    w = np.where(keep, np.exp(z - z.max()), 0.0)
    p = w / w.sum()
    if top_p < 1:
        order = np.argsort(-z, kind="stable")
        order = order[keep[order]]
        run = np.cumsum(p[order])
        many = int((run <= float(np.float32(top_p))).sum()) + 1
        p[order[many:]] = 0
        p /= p.sum()
    return p


def verify(logits, drafts, n, probs, u, temperature, top_k, top_p, greedy):
    """(accepted, next, p of the drafts) of one sequence."""
    pd = np.zeros(len(drafts))
    kept, alive = 0, True
    for i in range(n):
        if greedy:
            pd[i] = float(drafts[i] == int(logits[i].argmax()))
            ok = pd[i] > 0
        else:
            p = distribution(logits[i], temperature, top_k, top_p)
            x = drafts[i]
            pd[i] = p[x] if 0 <= x < p.size else 0.0
            q = 1.0 if probs is None else float(probs[i][x]) if 0 <= x < p.size else 0.0
            ok = float(u[i]) * q < pd[i]
        alive = alive and ok
        kept += alive
    if greedy:
        return kept, int(logits[kept].argmax()), pd
    p = distribution(logits[kept], temperature, top_k, top_p)
    if kept < n:
        q = probs[kept].astype(np.float64) if probs is not None else np.zeros_like(p)
        if probs is None and 0 <= drafts[kept] < p.size:
            q[drafts[kept]] = 2.0
        rest = np.maximum(p - q, 0.0)
        p = rest if rest.sum() > 0 else p
    run = np.cumsum(p)
    return kept, int(np.argmax(run > float(u[-1]) * run[-1])), pd


def check(S, logits, drafts, u, probs=None, n=None, temperature=1.0, top_k=0, top_p=1.0, do_sample=True, status=None):
    B, T = drafts.shape
    acc, nxt = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pd = torch.full((B, T), -9.0, device="cuda")
    ws = S.alloc_verify_workspace(B, T)
    kw = dict(uniform=u, draft_probs=probs, n_draft=n, p_draft=pd, temperature=temperature, top_k=top_k, top_p=top_p,
              do_sample=do_sample)
    S.verify_drafts(logits, drafts, acc, nxt, ws, **kw)
    assert S.workspace_status(ws) == (S.OK if status is None else status)
    greedy = not do_sample or temperature <= 0
    lg, dr, us = logits.float().cpu().numpy(), drafts.cpu().numpy(), u.cpu().numpy()
    pr = None if probs is None else probs.cpu().numpy()
    for b in range(B):
        nb = T if n is None else min(max(int(n[b]), 0), T)
        want = verify(lg[b], dr[b], nb, None if pr is None else pr[b], us[b], temperature, top_k, top_p, greedy)
        assert (int(acc[b]), int(nxt[b])) == want[:2], b
        # masses to 2^-43 of the row's largest, the sum to as many times the tokens' square root, one fp32
        # rounding (2^-24); probabilities are at most 1
        assert np.abs(pd[b].cpu().numpy() - want[2]).max() <= 2.0 ** -24 + 1e-10, b
    return acc, nxt


def case(B, T, V, seed, peak=6.0, spread=2.0, pad=0):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    base = spread * rnd(B, T + 1, V)
    base.scatter_add_(2, torch.randint(0, V, (B, T + 1, 8), generator=g, device="cuda"), peak * torch.rand(B, T + 1, 8, generator=g, device="cuda"))
    logits = torch.full((B, T + 1, V + pad), 30.0, device="cuda").to(torch.bfloat16)
    logits[..., :V] = base.to(torch.bfloat16)
    probs = torch.softmax(base[:, :T] + 0.7 * rnd(B, T, V), -1)
    drafts = torch.searchsorted(probs.cumsum(-1), torch.rand(B, T, 1, generator=g, device="cuda")).squeeze(-1).clamp_max(V - 1).to(torch.int32)
    return logits[..., :V], drafts, torch.rand(B, T + 1, generator=g, device="cuda"), probs


@pytest.mark.parametrize("V,pad", [(1, 0), (2, 0), (7, 0), (8, 0), (100, 3), (1001, 0), (4096, 0), (49152, 0), (65537, 6), (128257, 0)])
@pytest.mark.parametrize("kw", [dict(), dict(temperature=0.7), dict(top_k=5), dict(top_p=0.8), dict(temperature=1.3, top_k=40, top_p=0.9),
                                dict(top_p=0.0), dict(top_k=1), dict(do_sample=False)])
def test_against_the_definition(S, V, pad, kw):
    B, T = (6, 3) if V > 10000 else (16, 4)
    logits, drafts, u, probs = case(B, T, V, seed=V, pad=pad)
    check(S, logits, drafts, u, probs, **kw)
    check(S, logits, drafts, u, None, **kw)


@pytest.mark.parametrize("T", [1, 2, 33])
def test_ragged_drafts(S, T):
    B = 9
    logits, drafts, u, probs = case(B, T, 777, seed=T)
    n = torch.tensor([(i * 5) % (T + 1) for i in range(B)], dtype=torch.int32, device="cuda")
    check(S, logits, drafts, u, probs, n=n, top_k=30)
    check(S, logits, drafts, u, None, n=n, do_sample=False)


def test_flat_and_tied_rows(S):
    B, T, V = 8, 2, 5000
    _, drafts, u, probs = case(B, T, V, seed=1)
    flat = torch.zeros(B, T + 1, V, device="cuda", dtype=torch.bfloat16)
    few = (torch.arange(V, device="cuda") % 3).to(torch.bfloat16).expand(B, T + 1, V).contiguous()
    # cuts inside a group of equal values; goals next to a whole number of tokens are the definition's to
    # rounding, so top_p is kept away from those
    for logits in (flat, few, -few):
        for kw in (dict(), dict(top_k=1), dict(top_k=2500), dict(top_p=0.30001), dict(top_p=0.77777, top_k=3700)):
            check(S, logits, drafts, u, probs, **kw)
            check(S, logits, drafts, u, None, **kw)


@pytest.mark.parametrize("top_k", [1, 2, 7, 255, 256, 257, 511, 512, 513, 900])
@pytest.mark.parametrize("V", [600, 5003, 49152])
def test_filters_on_both_ways(S, V, top_k):
    """top-k around the sizes at which the row's work changes, few and many equal values among them."""
    B, T = 4, 2
    logits, drafts, u, probs = case(B, T, V, seed=V + top_k, spread=1.0)
    coarse = (logits.float() * 4).round().div(4).to(torch.bfloat16)       # many ties
    for lg in (logits, coarse, -logits.abs()):
        for kw in (dict(), dict(top_p=0.9), dict(top_p=0.3333, temperature=2.0)):
            check(S, lg, drafts, u, probs, top_k=top_k, **kw)
            check(S, lg, drafts, u, None, top_k=top_k, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=300), dict(top_k=100000, top_p=0.9), dict(top_p=0.5)])
def test_values_that_fill_a_counter(S, kw):
    """65,536 tokens and more of one value, of either sign, among 150,000."""
    V, T = 150000, 6
    logits, drafts, u, probs = case(2, T, V, seed=3)
    at = torch.randperm(V, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    for i, (many, value, other) in enumerate([(65535, 1.5, None), (65536, 1.5, None), (131072, -0.75, None), (70000, -0.75, 1.5),
                                              (65536, 0.0, -0.75), (65537, -9.0, 9.0), (150000, -3.0, None)]):
        logits[:, i, at[:many]] = value
        if other is not None:
            logits[:, i, at[many:many + 65536]] = other   # 65,536 of these too, where they fit
    check(S, logits, drafts, u, probs, **kw)
    check(S, logits, drafts, u, None, **kw)


@pytest.mark.parametrize("B", [2, 80])
@pytest.mark.parametrize("spread,peak,kw", [(400.0, 0.0, dict(temperature=60.0)), (2.0, 900.0, dict()), (300.0, 700.0, dict(top_p=0.9)),
                                            (5.0, 0.0, dict(temperature=50.0, top_k=300)), (0.5, 6.0, dict(top_p=0.7)),
                                            (400.0, 0.0, dict(temperature=90.0, top_k=700, top_p=0.8))])
def test_large_logits_and_temperatures(S, B, spread, peak, kw):
    logits, drafts, u, probs = case(B, 3, 3001, seed=8, spread=spread, peak=peak)
    check(S, logits, drafts, u, probs, **kw)
    check(S, logits, drafts, u, None, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=700, top_p=0.3), dict(top_k=3)])
def test_the_largest_vocabulary(S, kw):
    V, T = 2 ** 19, 2
    logits, drafts, u, probs = case(1, T, V, seed=6)
    logits[0, 0] = 1.0                                     # all equal: the largest sum, 2^63 units
    check(S, logits, drafts, u, probs, **kw)
    u[0, :2] = 1.0
    check(S, logits, drafts, u, None, **kw)
    logits[0, 2] = -2.5
    u[0, :2] = 0.0                                         # everything stays: the draw from the last row
    check(S, logits, drafts, u, probs, **kw)


@pytest.mark.parametrize("hidden", [-math.inf, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=300, top_p=0.9)])
def test_a_masked_vocabulary(S, hidden, kw):
    V, T = 128257, 3
    logits, drafts, u, probs = case(2, T, V, seed=5)
    logits[0, :, :100000] = hidden                         # all that is looked at first
    logits[1, :, 70:] = hidden
    drafts[1] = torch.tensor([69, 3, 128256])
    check(S, logits, drafts, u, probs, **kw)
    check(S, logits, drafts, u, None, **kw)


def test_zeros_of_both_signs_are_equal(S):
    B, T, V = 12, 2, 3000
    g = torch.Generator("cuda").manual_seed(21)
    _, drafts, u, probs = case(B, T, V, seed=7)
    logits = torch.randint(-1, 2, (B, T + 1, V), generator=g, device="cuda").float()
    logits = torch.where(torch.rand(logits.shape, generator=g, device="cuda") < 0.5, -logits.abs().neg(), logits * 0.0)
    logits = (logits * torch.where(torch.rand(logits.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)).to(torch.bfloat16)
    assert bool((torch.signbit(logits) & (logits == 0)).any()) and bool((~torch.signbit(logits) & (logits == 0)).any())
    for kw in (dict(), dict(top_k=1500), dict(top_p=0.66666), dict(top_p=0.5001, top_k=2000)):
        check(S, logits, drafts, u, probs, **kw)
    check(S, torch.where(logits > 0, -logits, logits), drafts, u, None, do_sample=False)   # the zeros are the maximum


def test_masked_and_extreme_logits(S):
    B, T, V = 6, 3, 3000
    logits, drafts, u, probs = case(B, T, V, seed=2)
    masked = logits.clone()
    masked[:, :, 100:2900] = -math.inf
    check(S, masked, drafts, u, probs)
    check(S, masked, drafts, u, probs, top_k=500, top_p=0.95)
    lowest = logits.clone()
    lowest[:, :, ::2] = torch.finfo(torch.bfloat16).min
    check(S, lowest, drafts, u, probs)
    check(S, lowest, drafts, u, None, top_k=2000)
    check(S, logits * 1000, drafts, u, probs)
    check(S, logits * 1e-6, drafts, u, probs)
    check(S, logits - 200, drafts, u, probs, top_p=0.9)        # every value negative
    check(S, logits + 200, drafts, u, probs, top_p=0.9)
    check(S, logits, drafts, u, probs, temperature=100.0)
    check(S, logits, drafts, u, probs, temperature=0.01)
    check(S, logits, drafts, u, probs, temperature=1e-39)      # its reciprocal is infinite in 32 bits


def test_equal_distributions_keep_everything(S):
    # q is p as far as 32 bits go and u < 1: every draft stays; u next to 1 takes the last of the row
    B, T, V = 5, 4, 2000
    logits, drafts, u, _ = case(B, T, V, seed=3)
    q = torch.softmax(logits[:, :T].float(), -1)
    u = u * 0.999
    u[:, -1] = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24], device="cuda")
    acc, _ = check(S, logits, drafts, u, q)
    assert bool((acc == T).all())


def test_nothing_left_of_the_difference(S):
    # a drafter whose "probabilities" are above the target's everywhere: the draw falls back to p
    B, T, V = 4, 2, 300
    logits, drafts, u, _ = case(B, T, V, seed=4)
    u[:, :T] = 0.9999
    acc, _ = check(S, logits, drafts, u, torch.full((B, T, V), 1.5, device="cuda"))
    assert bool((acc == 0).all())


def test_bad_inputs_are_recorded(S):
    B, T, V = 3, 2, 500
    logits, drafts, u, probs = case(B, T, V, seed=5)
    bad = drafts.clone()
    bad[1, 0], bad[2, 1] = V, -1
    for kw in (dict(probs=probs), dict(), dict(do_sample=False)):
        check(S, logits, bad, u, status=S.ERR_INPUT, **kw)
    n = torch.tensor([2, 5, -1], dtype=torch.int32, device="cuda")
    check(S, logits, drafts, u, probs, n=n, status=S.ERR_INPUT)
    for value in (math.nan, math.inf, -math.inf):
        row = logits.clone()
        row[1, 0] = value
        acc, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        ws = S.alloc_verify_workspace(B, T)
        for do_sample in (True, False):
            S.verify_drafts(row, drafts, acc, nxt, ws, uniform=u, draft_probs=probs, do_sample=do_sample)
            assert S.workspace_status(ws) == S.ERR_INPUT
            assert int(acc[1]) == 0 and int(nxt[1]) == -1 and 0 <= int(nxt[0]) < V


def test_frequencies_follow_the_target(S):
    """The first emitted token of many sequences with one target row and one drafter: its counts are the
    target's probabilities to within five standard deviations."""
    V, B = 12, 40000
    g = torch.Generator("cuda").manual_seed(11)
    row = torch.randn(2, V, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.softmax(torch.randn(V, generator=g, device="cuda"), -1)
    drafts = torch.searchsorted(q.cumsum(-1), torch.rand(B, 1, generator=g, device="cuda")).clamp_max(V - 1).to(torch.int32)
    u = torch.rand(B, 2, generator=g, device="cuda")
    acc, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = S.alloc_verify_workspace(B, 1)
    S.verify_drafts(row.expand(B, 2, V).contiguous(), drafts, acc, nxt, ws, uniform=u, draft_probs=q.expand(B, 1, V).contiguous())
    first = torch.where(acc == 1, drafts[:, 0], nxt)
    p = torch.softmax(row[0].double(), -1)
    count = torch.bincount(first.long(), minlength=V).double()
    assert bool(((count - B * p).abs() <= 5 * (B * p * (1 - p)).sqrt()).all())


def test_tensors_of_another_device_are_refused(S, monkeypatch):
    logits, drafts, u, probs = case(1, 2, 100, seed=7)
    acc, nxt = (torch.full((1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = S.alloc_verify_workspace(1, 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: logits.device.index + 1)
    with pytest.raises(ValueError, match="current device"):
        S.verify_drafts(logits, drafts, acc, nxt, ws, uniform=u, draft_probs=probs)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert int(acc) == -9 and int(nxt) == -9


@pytest.mark.parametrize("top", [10.0, 27.75, 31.0, 31.5])
def test_a_long_tail_of_one_error(S, top):
    """One likely token behind (V - 1) equal ones, whose masses are rounded alike (31.0: to twice of what they are,
    nearly) or fall below half a unit (31.5).  Every draw's border is within the header's V * 2^-45 of the definition's."""
    V, B = 128257, 64
    logits = torch.zeros(B, 2, V, device="cuda", dtype=torch.bfloat16)
    logits[:, :, V - 1] = top
    tail = (V - 1) / (V - 1 + math.exp(top))                # what the equal tokens have of the whole
    u = torch.rand(B, 2, generator=torch.Generator("cuda").manual_seed(9), device="cuda")
    u[:32, 1] = (torch.linspace(0.0, 2.0, 32, device="cuda") * tail).clamp_max(1 - 2.0 ** -24)   # among them, and around their end
    drafts = torch.full((B, 1), V - 1, dtype=torch.int32, device="cuda")
    acc, nxt = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pd, ws = torch.zeros(B, 1, device="cuda"), S.alloc_verify_workspace(B, 1)
    S.verify_drafts(logits, drafts, acc, nxt, ws, uniform=u, p_draft=pd)
    assert S.workspace_status(ws) == S.OK
    bound = V * 2.0 ** -45
    p = 1.0 - tail
    assert bool(((pd.double() - p).abs() <= 2.0 ** -24 + bound).all())
    for b in range(B):
        u0, u1, x = float(u[b, 0]), float(u[b, 1]), int(nxt[b])
        if abs(u0 - p) > bound:
            assert int(acc[b]) == int(u0 < p)
        if int(acc[b]) == 1:                                # drawn from the row
            below, upto = tail * x / (V - 1), 1.0 if x == V - 1 else tail * (x + 1) / (V - 1)
        else:                                               # the draft is gone: drawn from the equal ones
            assert x < V - 1
            below, upto = x / (V - 1), (x + 1) / (V - 1)
        assert below - bound <= u1 < upto + bound, (b, x, u1)
