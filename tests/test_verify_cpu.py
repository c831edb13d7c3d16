"""Host-side refusals of smol_verify_drafts (no GPU needed)."""
import pytest
import torch

from llama_decoder_forward_gb300 import build as B

P = 0x10000


@pytest.fixture(scope="module")
def S():
    B.build()
    from llama_decoder_forward_gb300 import smol
    return smol


def call(S, **kw):
    a = dict(logits=P, ld=100, drafts=P, n_draft=None, probs=P, ldq=100, B=4, T=3, V=100, temperature=1.0, top_k=0, top_p=1.0,
             do_sample=1, uniform=P, n_accepted=P, next=P, p_draft=P, ws=P, n=1 << 30, stream=None)
    a.update(kw)
    return S.raw.smol_verify_drafts(*a.values())


def test_refusals(S):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(logits=None), dict(drafts=None), dict(n_accepted=None), dict(next=None), dict(ws=None), dict(uniform=None),
               dict(B=0), dict(T=0), dict(V=0), dict(ld=99), dict(ldq=99), dict(temperature=nan), dict(top_p=nan), dict(temperature=inf)):
        assert call(S, **kw) == -1, kw
    for kw in (dict(V=(1 << 19) + 1, ld=1 << 20, ldq=1 << 20), dict(B=1 << 24, T=1), dict(T=513)):
        assert call(S, **kw) == -2, kw
    for kw in (dict(logits=P + 1), dict(drafts=P + 2), dict(n_draft=P + 1), dict(probs=P + 2), dict(uniform=P + 1), dict(next=P + 3),
               dict(n_accepted=P + 1), dict(p_draft=P + 2), dict(ws=P + 8)):
        assert call(S, **kw) == -3, kw
    assert call(S, n=100) == -5
    # greedy needs no random numbers: on to the next check
    assert call(S, do_sample=0, uniform=None, n=100) == -5 and call(S, temperature=0.0, uniform=None, n=100) == -5
    assert S.last_launch_count() == 0


def test_workspace_query(S):
    size = S.raw.smol_verify_workspace_bytes
    assert size(4, 3) >= 1024 + 16 * 8 and size(0, 3) == 0 and size(4, 0) == 0 and size(1 << 24, 1) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused must find no device: the addresses are made up")
def test_outputs_on_inputs_are_refused(S):
    """The CTAs of a sequence read its inputs at their own time: none may see another's outputs there."""
    B, T = 4, 3
    apart = dict(B=B, T=T, drafts=P, n_draft=P + 0x1000, uniform=P + 0x2000, n_accepted=P + 0x3000, next=P + 0x4000,
                 p_draft=P + 0x5000, ws=P + 0x6000, logits=P + 0x100000, probs=P + 0x200000)
    for out in ("n_accepted", "next", "p_draft", "ws"):
        for other in ("drafts", "n_draft", "uniform", "n_accepted", "next", "p_draft"):
            if other != out:
                assert call(S, **dict(apart, **{out: apart[other]})) == -1, (out, other)
    assert call(S, **dict(apart, next=apart["drafts"] + 4 * (B * T - 1))) == -1            # the last draft
    assert call(S, **dict(apart, p_draft=apart["uniform"] - 4 * (B * T - 1))) == -1
    assert call(S, **dict(apart, n_accepted=apart["uniform"] + 4 * (B * (T + 1) - 1))) == -1
    assert S.last_launch_count() == 0
    # side by side is apart, and a greedy call reads no random numbers: on to the launch, for which there is no device
    for kw in (dict(next=apart["drafts"] + 4 * B * T), dict(n_accepted=apart["drafts"] - 4 * B),
               dict(do_sample=0, p_draft=apart["uniform"])):
        assert call(S, **dict(apart, **kw)) not in (-1, -3, -5), kw
