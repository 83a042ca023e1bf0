"""CPU checks of the lists that gradient norm and clipping take: an output shares memory with no other
tensor, in any arrangement, and everything else serves."""
import itertools

import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16


def views(*spans, dtype=F32):
    """Views of one buffer, from and to the given elements."""
    flat = torch.zeros(200, dtype=dtype)
    return [flat[a:b] for a, b in spans]


def refused(m, grads, out=None):
    with pytest.raises(ValueError, match="same memory"):
        m._grad_list(grads, out)


def test_swapped_outputs(mxq_lib):
    a, b, c = torch.zeros(10), torch.zeros(10), torch.zeros(10)
    refused(mxq_lib, [a, b], [b, a])
    refused(mxq_lib, [a, b, c], [b, c, a])
    refused(mxq_lib, [a, b], [b, c])           # written before or after it is read
    refused(mxq_lib, [b, a], [c, b])
    mxq_lib._grad_list([a], [b])


def test_an_output_beside_its_own_gradient(mxq_lib):
    for shift in (1, 5, 9):
        g, o, far = views((20, 30), (20 + shift, 30 + shift), (40, 50))
        refused(mxq_lib, [g], [o])
        refused(mxq_lib, [o], [g])
    g, o = views((20, 30), (30, 40))
    mxq_lib._grad_list([g], [o])
    mxq_lib._grad_list([g], [g])
    mxq_lib._grad_list([g], [g.view(10)])      # another tensor of the same memory is in place too
    # the bytes count, not the elements
    flat = torch.zeros(40, dtype=BF16)
    wide = flat.view(F32)
    refused(mxq_lib, [flat[:10]], [wide[4:14]])
    mxq_lib._grad_list([flat[:10]], [wide[5:15]])


def test_parts_of_another(mxq_lib):
    whole, part, end, beside = views((0, 100), (30, 40), (99, 109), (100, 110))
    for grads in itertools.permutations([whole, part]):
        refused(mxq_lib, list(grads))
    refused(mxq_lib, [whole, end])
    refused(mxq_lib, [part, whole, beside])
    mxq_lib._grad_list([whole, beside])
    elsewhere = [torch.zeros(t.numel()) for t in (whole, part)]
    mxq_lib._grad_list([whole, part], elsewhere)             # what is only read may be the same
    mxq_lib._grad_list([whole, whole], [torch.zeros(100), torch.zeros(100)])
    refused(mxq_lib, [elsewhere[1], elsewhere[0]], [part, whole])
    refused(mxq_lib, [whole, elsewhere[1]], [elsewhere[0], part])   # a gradient that another's output is part of
    # a long one in front, a short one behind it, then one that the long one reaches
    a, b, c = views((0, 100), (100, 120), (50, 60))
    refused(mxq_lib, [a, b, c])
    refused(mxq_lib, [torch.zeros(20), a, torch.zeros(10)], [b, torch.zeros(100), c])
    assert [v.g for v in mxq_lib._grad_list([a, c, a], write=False)[0]] == [a.data_ptr(), c.data_ptr(), a.data_ptr()]


def test_every_arrangement_of_three(mxq_lib):
    """Two gradients and one output of three elements each, anywhere in a buffer of seven, against the definition."""
    flat, other = torch.zeros(7), torch.zeros(3)
    for p, q, r in itertools.product(range(5), repeat=3):
        g, h, o = flat[p:p + 3], flat[q:q + 3], flat[r:r + 3]
        bad = (abs(p - r) < 3 and p != r) or abs(q - r) < 3
        try:
            mxq_lib._grad_list([g, h], [o, other])
            assert not bad, (p, q, r)
        except ValueError as e:
            assert bad and "same memory" in str(e), (p, q, r)


def test_messages_name_the_output(mxq_lib):
    a, b, c = views((0, 10), (5, 15), (50, 60))
    with pytest.raises(ValueError, match="output 1: in the same memory as output 0"):
        mxq_lib._grad_list([a, b])
    for grads, out in (([c, b], [a, torch.zeros(10)]), ([c, a], [b, torch.zeros(10)])):
        with pytest.raises(ValueError, match="output 0: in the same memory as gradient 1"):
            mxq_lib._grad_list(grads, out)


def test_empty_tensors_share_with_nobody(mxq_lib):
    a, none, empty = views((0, 10), (5, 5), (0, 0))
    mxq_lib._grad_list([a, none, empty, empty])
    mxq_lib._grad_list([none, empty], [a[3:3], a[3:3]])
