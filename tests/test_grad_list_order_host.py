"""CPU checks of the order of elements in gradient lists: an output has its gradient's, and the strides of
dimensions of one element say nothing about it."""
import pytest
import torch


def test_one_element_dimensions(mxq_lib):
    m = mxq_lib
    for shape, one, two in (((1, 5), (5, 1), (77, 1)), ((5, 1), (1, 1), (1, 5)), ((4, 1, 3), (3, 3, 1), (3, 99, 1)),
                            ((1, 1), (1, 1), (8, 3)), ((1,), (1,), (4,)), ((3, 4, 1), (1, 3, 12), (1, 3, 1))):
        g, o = torch.empty_strided(shape, one), torch.empty_strided(shape, two)
        for a, b in ((g, o), (o, g)):
            arr, _ = m._grad_list([a], [b])
            assert (arr[0].g, arr[0].out, arr[0].n) == (a.data_ptr(), b.data_ptr(), a.numel())


def test_no_elements(mxq_lib):
    g, o = torch.empty_strided((0, 4), (4, 1)), torch.empty_strided((0, 4), (1, 0))
    arr, _ = mxq_lib._grad_list([g], [o])
    assert arr[0].n == 0


def test_other_orders_are_refused(mxq_lib):
    for shape, one, two in (((3, 4), (4, 1), (1, 3)), ((3, 1, 4), (4, 4, 1), (1, 1, 3)), ((2, 3, 4), (12, 4, 1), (12, 1, 3))):
        g, o = torch.empty_strided(shape, one), torch.empty_strided(shape, two)
        for a, b in ((g, o), (o, g)):
            with pytest.raises(ValueError, match="output 0: shape"):
                mxq_lib._grad_list([a], [b])
    with pytest.raises(ValueError, match="output 0: shape"):
        mxq_lib._grad_list([torch.zeros(1, 5)], [torch.zeros(5)])
