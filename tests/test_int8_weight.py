"""Int8Weight's descriptor follows the weight it describes (no GPU: stand-ins for the tensors)."""
import pytest
import torch

import bit_nf4_quantized_nibble_amd as qn


class OnGpu:
    """What a descriptor reads of a tensor, with the storage of a CPU tensor in place of one on the GPU."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, t):
        self.t = t

    shape = property(lambda self: self.t.shape)
    dtype = property(lambda self: self.t.dtype)

    def data_ptr(self):
        return self.t.data_ptr()

    def is_contiguous(self):
        return self.t.is_contiguous()


def weight(rows=8, cols=16, experts=1):
    return qn.Int8Weight(rows, cols, OnGpu(torch.zeros(experts, rows, 128, dtype=torch.int8)),
                         OnGpu(torch.zeros(experts, rows)))


def test_the_descriptor_is_kept_while_nothing_changes():
    w = weight()
    assert w.descriptor() is w.descriptor()


def test_replaced_storages_are_followed():
    w = weight()
    assert w.descriptor().codes == w.codes.data_ptr()
    kept = w.codes.t, w.scale.t  # alive, so that no new storage can lie where they do
    w.codes.t = torch.ones(1, 8, 128, dtype=torch.int8)
    assert w.codes.data_ptr() != kept[0].data_ptr() and w.descriptor().codes == w.codes.data_ptr()
    w.scale.t = torch.ones(1, 8)
    assert w.scale.data_ptr() != kept[1].data_ptr() and w.descriptor().scale == w.scale.data_ptr()


def test_a_changed_tensor_is_checked_again():
    for change in (lambda w: setattr(w.codes, "t", w.codes.t[:, :4]), lambda w: setattr(w.scale, "t", w.scale.t[:, :4]),
                   lambda w: setattr(w.codes, "t", w.codes.t.view(torch.uint8)),
                   lambda w: setattr(w.scale, "t", w.scale.t.view(torch.int32)),
                   lambda w: setattr(w.codes, "t", w.codes.t.as_strided((1, 8, 128), (1024, 1, 8)))):
        w = weight()
        w.descriptor()
        change(w)
        with pytest.raises(ValueError):
            w.descriptor()


def test_changed_fields_are_checked_again():
    for rows, cols in ((4, 16), (9, 16), (8, 129), (8, 300)):
        w = weight()
        w.descriptor()
        w.rows, w.cols = rows, cols
        with pytest.raises(ValueError):
            w.descriptor()
    w = weight()
    w.descriptor()
    w.cols = 100  # as many stored columns: the descriptor says what the weight says
    assert w.descriptor().cols == 100


def test_experts_follow_the_codes():
    w = weight(experts=3)
    assert w.descriptor().experts == 3
    w.codes, w.scale = weight(experts=2).codes, weight(experts=2).scale
    assert w.descriptor().experts == 2
