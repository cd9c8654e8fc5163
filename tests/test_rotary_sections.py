"""Sections that rotary_axes refuses through its Python entry point: every entry 0 or
more and below 2^31, 1 to ROTARY_MAX_AXES of them. The sections are looked at before the tensors'
device, so that this needs no GPU; with tensors on one the same calls are refused."""
import pytest
import torch

import bit_quantized_gemm_amd as w4

BAD = [(8, -2), (-2,), (8, -1), (-1, 8), (-5, 8), (8, 2**31), (2**31, 8), (8, 2**80), (8, -2**80), (8, 0, -3, 4)]


def call(sections, device):
    x = torch.zeros(1, 2, 1, 32, dtype=torch.bfloat16, device=device)
    pos = torch.zeros(1, 2, len(sections), dtype=torch.int32, device=device)
    return w4.rotary_axes(x, pos, torch.ones(8, device=device), sections)


@pytest.mark.parametrize("sections", BAD, ids=str)
def test_refused(sections):
    with pytest.raises(ValueError, match="sections"):
        call(sections, "cpu")


@pytest.mark.parametrize("sections", [(), (1, 1, 1, 1, 1), (1, 1, 1, 1, -7)], ids=str)
def test_number_of_axes(sections):
    with pytest.raises(ValueError, match="axes"):
        call(sections, "cpu")


@pytest.mark.parametrize("sections", [(2.5,), ("2",), (8, None)], ids=str)
def test_not_whole_numbers(sections):
    with pytest.raises(TypeError):
        call(sections, "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("sections", BAD, ids=str)
def test_refused_with_device_tensors(sections):
    with pytest.raises(ValueError, match="sections"):
        call(sections, "cuda")
