"""Host-side refusals of smol_verify_drafts (no GPU needed)."""
import pytest

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
