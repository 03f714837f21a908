"""What the paged-cache calls of the binding take as rows of tokens (no GPU needed: the
tensors lie on the CPU, and so does the cache that they are compared with)."""
from types import SimpleNamespace

import pytest
import torch

from bit_group_quantized_qgemv_gb300 import _binding as b

CACHE = SimpleNamespace(index=-1, device="cpu", head_dim=64)


@pytest.mark.parametrize("make,want", [
    (lambda x: x(5, 3 * 64), (5, 192, 192)),
    (lambda x: x(5, 3, 64), (5, 192, 192)),
    (lambda x: x(5, 7, 64)[:, 2:5], (5, 192, 448)),
    (lambda x: x(5, 448)[:, 64:256], (5, 192, 448)),
    (lambda x: x(1, 448)[:, :192], (1, 192, 192)),        # the stride of a single row says nothing
    (lambda x: x(2, 5, 64).transpose(0, 1)[:, :1], (5, 64, 64)),   # nor that of a single head
    (lambda x: x(1, 5, 64).transpose(0, 1), (5, 64, 64)),
    (lambda x: x(0, 3, 64), (0, 192, 192)),
])
def test_rows_that_are_taken(make, want):
    t = make(lambda *s: torch.zeros(*s, dtype=torch.float16))
    assert b._token_rows(CACHE, t, "q") == (t.data_ptr(), *want)


@pytest.mark.parametrize("make", [
    lambda x: x(2, 5, 64).transpose(0, 1),                # heads apart
    lambda x: x(5, 64, 3).transpose(1, 2),
    lambda x: x(5, 384)[:, ::2],
    lambda x: x(192),
    lambda x: x(1, 5, 3, 64),
])
def test_rows_that_are_refused(make):
    with pytest.raises(ValueError):
        b._token_rows(CACHE, make(lambda *s: torch.zeros(*s, dtype=torch.float16)), "q")


def test_types_and_sizes():
    with pytest.raises(TypeError):
        b._token_rows(CACHE, torch.zeros(5, 64), "q")
    x = torch.zeros(5, 64, dtype=torch.float16)
    for rows, width in ((4, 64), (5, 128)):
        with pytest.raises(ValueError):
            b._token_rows(CACHE, x, "q", rows, width)
