"""The operators around verification together: a draft head distilled from
the target's top logits proposes tokens under truncated sampling, and more of
them are accepted than before it was trained."""
import pytest
import torch

from draft_verification_row_gb300 import draft_training as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def test_distilled_drafts_are_accepted_more_often():
    r = D.run(steps=60, rows=512, B=128, L=4, V=2000, d=64, rank=32)
    assert r["losses"][-1] < 0.5 * r["losses"][0], r
    assert r["accepted_after"] > r["accepted_before"] + 0.5, r


def test_a_draft_head_equal_to_the_target_is_accepted_whole():
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(3)
    lm_head = torch.randn((64, 3000), generator=g, device=dev) * 0.3
    head = lambda h: D.target_rows(h, lm_head)  # noqa: E731
    out, status = D.verify_drafts(head, torch.randn((32, 5, 64), generator=g, device=dev), lm_head,
                                  D.Sampling(top_k=20, top_p=0.9, min_p=0.02))
    assert int(status.item()) == 0
    # GBV's acceptance probability is 1 where both distributions are equal, up to fp32 rounding of the residual
    assert (out["accept_len"].float().mean() > 3.9)
