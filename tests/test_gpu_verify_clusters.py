"""zf_verify_drafts with 1, 2, 4, 8 and 16 CTAs per request: refused drafts sampled from the difference, from the target
itself where the difference is nowhere positive (the cluster sums its row again), and accepted ones."""
import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("vocab", [4095, 4096, 8192, 16385, 16388, 32768, 50001])
def test_every_cluster_size(vocab, with_draft):
    zf = H.zf_module()
    B, T = 6, 2
    g = torch.Generator().manual_seed(vocab)
    target = torch.softmax(torch.randn(B, T + 1, vocab, generator=g), -1)
    draft = torch.softmax(torch.randn(B, T, vocab, generator=g), -1)
    drafts = torch.randint(0, vocab, (B, T), generator=g).to(torch.int32)
    uniform = torch.rand(B, T + 1, generator=g)
    uniform[:, :T] = 1 - 2.0 ** -24                        # refused but where q is no larger than p
    draft[1] = 2 * target[1, :T]                           # refused at once, p nowhere above q
    target[2, 1] = 0                                       # the second draft: nothing to sample, from either
    draft[2, 0, drafts[2, 0]] = target[2, 0, drafts[2, 0]] / 2
    target[3, 0] = 0                                       # all of the mass on a refused draft: the row itself
    target[3, 0, drafts[3, 0]] = 0.5
    draft[3, 0, drafts[3, 0]] = 1
    uniform[4, :T] = 0                                     # accepted
    uniform[5, 0] = 0                                      # the first accepted only
    draft = draft if with_draft else None
    acc, tok, gaps, st = S.verify(target.numpy(), None if draft is None else draft.numpy(), drafts.numpy(), None, uniform.numpy())
    assert min(gaps) > 2.0 ** -44 and acc[4] == T and acc[3] == 0 and tok[3][0] == drafts[3, 0]
    args = [t.cuda() for t in (target, drafts, uniform)]
    draft = None if draft is None else draft.cuda()
    for batch in (B, 1):                                   # (fewer requests: larger clusters)
        for b in range(0, B, batch):
            part = [x[b:b + batch].contiguous() for x in args]
            for _ in range(10):
                a, t = zf.verify_drafts(*part, draft_probs=None if draft is None else draft[b:b + batch].contiguous())
                assert a.tolist() == acc[b:b + batch] and t.tolist() == tok[b:b + batch]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    zf.verify_drafts(*args, draft_probs=draft, status=status)
    assert int(status) == st
