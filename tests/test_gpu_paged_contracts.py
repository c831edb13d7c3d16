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
