"""What the binding asks of MXFP4 operands and of streams (CPU only): the row
count of a call is the pitch of the panels that it reads, and a stream belongs
to the tensors' device."""
import types

import pytest
import torch

ns = pytest.importorskip("newton_schulz_amd")


def _operand(panels, rows):
    return torch.zeros(panels, rows, 128, dtype=torch.uint8), torch.zeros(panels, rows, 8, dtype=torch.uint8)


def test_operands_of_the_stated_shape():
    ns._need_mx(*_operand(3, 70), "x", 70, 600)
    codes, scales = _operand(3, 70)
    ns._need_mx(codes.view(-1), scales.view(-1), "x", 70, 600)                   # flat buffers
    ns._need_mx(codes.view(-1, 128), scales.view(-1, 8), "x", 70, 600)           # a row a line
    ns._need_mx(torch.zeros(3 * 70 * 128 + 64, dtype=torch.uint8), scales, "x", 70, 600)     # with room behind


@pytest.mark.parametrize("rows,cols", [(64, 600), (69, 600), (71, 600), (70, 500), (70, 800)])
def test_operands_of_another_shape_are_refused(rows, cols):
    codes, scales = _operand(3, 70)
    with pytest.raises(ValueError):
        ns._need_mx(codes, scales, "x", rows, cols)
    with pytest.raises(ValueError):
        ns._need_mx(codes, torch.zeros(3 * 71 * 8, dtype=torch.uint8), "x", rows, cols)
    right = _operand(ns._mx_panels(cols), rows)
    with pytest.raises(ValueError):
        ns._need_mx(right[0], scales, "x", rows, cols)
    with pytest.raises(ValueError):                     # the right size, rows first
        ns._need_mx(right[0].transpose(0, 1).contiguous(), right[1], "x", rows, cols)
    with pytest.raises(ValueError):
        ns._need_mx(codes.view(-1, 128), right[1], "x", rows, cols)


def test_a_stream_of_another_device_is_refused():
    """Also where the caller gives every output and the workspace."""
    dev = torch.device("cuda", 0)
    here = types.SimpleNamespace(cuda_stream=64, device=dev)
    assert ns._stream(here, dev).value == 64
    assert ns._stream(types.SimpleNamespace(cuda_stream=64), dev).value == 64        # any holder of a handle
    with pytest.raises(ValueError):
        ns._stream(types.SimpleNamespace(cuda_stream=64, device=torch.device("cuda", 1)), dev)
