"""Lengths that zf_verify_drafts shortens by more than they hold."""
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [40, 5001, 32000])
def test_lengths_do_not_fall_below_zero(vocab):
    """Requests shorter than their refused drafts end at 0, and the status word says so."""
    zf = H.zf_module()
    T, lens = 3, [50, 2, 0, 1]
    B = len(lens)
    g = torch.Generator().manual_seed(vocab)
    target = torch.softmax(torch.randn(B, T + 1, vocab, generator=g), -1)
    drafts = torch.randint(0, vocab, (B, T), generator=g).to(torch.int32)
    uniform = 0.5 + 0.5 * torch.rand(B, T + 1, generator=g)
    acc, tok, gaps, _ = S.verify(target.numpy(), None, drafts.numpy(), None, uniform.numpy())
    assert min(gaps) > 2.0 ** -44 and acc == [0] * B              # (no target puts half its mass on one token)
    status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    a, t = zf.verify_drafts(target.cuda(), drafts.cuda(), uniform.cuda(), seq_lens=out, new_seq_lens=out, status=status)
    assert a.tolist() == acc and t.tolist() == tok
    assert out.tolist() == [47, 0, 0, 0] and int(status) == S.DEV_BAD_SEQ_LEN
