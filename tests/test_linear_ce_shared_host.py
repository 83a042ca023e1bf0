"""CPU checks of the memory that mxq_linear_ce_backward's outputs may be in: none of another tensor's, where columns of
one buffer that lie between each other have nothing in common."""
import itertools

import pytest
import torch


def bytes_of(t):
    at = t.data_ptr() + torch.arange(t.shape[0])[:, None] * (t.stride(0) * t.element_size()) if t.dim() == 2 else torch.tensor([[t.data_ptr()]])
    wide = (t.shape[1] if t.dim() == 2 else t.numel()) * t.element_size()
    return set((at + torch.arange(wide)).flatten().tolist())


def test_share_against_every_byte(mxq_lib):
    flat = torch.zeros(400, dtype=torch.bfloat16)
    views = [flat.as_strided((rows, cols), (ld, 1), at) for rows, cols, ld in ((1, 30, 30), (3, 8, 8), (3, 8, 20), (4, 12, 20), (5, 4, 16), (2, 40, 64), (1, 1, 1), (3, 0, 8))
             for at in (0, 3, 8, 12, 20, 41, 100)]
    views += [torch.zeros(40), flat[5:25], flat.view(torch.int32)[10:20]]
    seen = [bytes_of(v) if v.numel() else set() for v in views]
    both = 0
    for (a, sa), (b, sb) in itertools.product(list(zip(views, seen)), repeat=2):
        assert mxq_lib._share(a, b) == bool(sa & sb), (a.shape, a.stride(), a.storage_offset(), b.shape, b.stride(), b.storage_offset())
        both += bool(sa & sb)
    assert both > 500


def test_refused(mxq_lib):
    x, w, t, s = torch.zeros(4, 64), torch.zeros(9, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2)
    ok = dict(dx=torch.zeros(4, 64), dw=torch.zeros(9, 64), x=x, w=w, targets=t, stats=s, weight=None)
    mxq_lib._refuse_shared(**ok)
    mxq_lib._refuse_shared(**{**ok, "dx": None, "dw": None})
    for name, other in (("dx", x), ("dw", w), ("dx", w[:4]), ("dw", w.view(-1)[:576].view(9, 64))):
        with pytest.raises(ValueError, match=f"{name}: in the same memory as"):
            mxq_lib._refuse_shared(**{**ok, name: other})
    both = torch.zeros(12, 64)
    with pytest.raises(ValueError, match="dx: in the same memory as dw"):
        mxq_lib._refuse_shared(**{**ok, "dx": both[:4], "dw": both[3:]})
    mxq_lib._refuse_shared(**{**ok, "dx": both[:3], "dw": both[3:]})
