"""zf_verify_mapped_drafts without a GPU: what it refuses before anything is launched, in the C ABI and in the
binding, and pins of its oracle."""
import numpy as np
import pytest
import torch

from oracle import zf_step_oracle as S
from tests import helpers as H


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


def test_mapped_verify_refuses(zf):
    f = zf.lib().zf_verify_mapped_drafts
    names = ["batch", "drafts", "vocab", "target", "draft", "tokens", "n", "uniform", "start", "accepted", "out", "lens",
             "new_lens", "status", "stream"]
    good = [2, 3, 100, 0x1000, 0x2000, 0x3000, 0x3100, 0x3200, 0x3500, 0x3300, 0x3400, None, None, None, None]

    def call(**kw):
        args = list(good)
        for k, v in kw.items():
            args[names.index(k)] = v
        return f(*args)
    for kw in (dict(batch=-1), dict(batch=4097), dict(drafts=0), dict(drafts=65), dict(vocab=0), dict(start=None),
               dict(start=0x3502), dict(lens=0x4000), dict(target=None), dict(accepted=None), dict(out=None), dict(draft=0x2001)):
        assert call(**kw) == -1, kw
    assert call(batch=0) == 0 and call(batch=0, start=None) == 0


def test_binding_checks_token_start(zf):
    p, d, u = torch.zeros(2, 4, 9), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4)
    start = torch.zeros(3, dtype=torch.int32)
    for x, msg in ((start[:2], "token_start: shape"), (start.long(), "token_start: dtype"),
                   (start.to("meta"), "token_start is on meta"), (start, "a CUDA device")):
        with pytest.raises(ValueError, match=msg):
            zf.verify_drafts(p, d, u, token_start=x)
    with pytest.raises(TypeError, match="token_start"):
        zf.verify_drafts(p, d, u, token_start=[0, 4, 8])


def test_oracle_step_pins():
    p = np.array([[[0.5, 0.5, 0.0], [0.1, 0.2, 0.7]]], np.float32).repeat(3, 0)
    drafts, u = np.array([[1], [1], [2]]), np.array([[0.6, 0.9], [0.6, 0.9], [0.6, 0.2]], np.float32)
    # refused (0.6 >= 0.5): the place of the draft is taken off; nothing mapped: nothing happens
    acc, tok, lens, _, st = S.verify_step(p, None, drafts, None, u, [0, 2, 2, 4], [9, 7, 0])
    assert acc == [0, 0, 0] and tok == [[0, -1], [-1, -1], [0, -1]] and lens == [8, 7, 0] and st == S.DEV_BAD_SEQ_LEN
    acc, tok, lens, _, st = S.verify_step(p[:1], None, drafts[:1], None, u[:1], [0, 3], [9])
    assert acc == [0] and tok == [[-1, -1]] and lens == [9] and st == S.DEV_BAD_DRAFT
    # two drafts' places, one draft: the place behind it goes too
    acc, tok, lens, _, st = S.verify_step(p[:1].repeat(2, 1)[:, :3], None, np.array([[1, 1]]), [1], np.array([[0.1, 0.1, 0.9]], np.float32),
                                          [0, 3], [9])
    assert acc == [1] and lens == [8] and st == 0
