"""Rare inputs of the paged-cache operators: rows that the caller masks, weights far below
a row's largest, positions at the end of the 32-bit range, starts and lengths out of range
where no token lies."""
import math

import pytest
import torch

import kv_reference as ref
from test_gpu_kv_cache import close, handle, queries

pytestmark = pytest.mark.gpu

q = pytest.importorskip("bit_group_quantized_qgemv_gb300")


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("n_q,n_kv,m", [(4, 1, 5), (8, 1, 4), (4, 4, 20), (4, 1, 20), (6, 2, 40), (2, 2, 200),
                                        (8, 1, 90), (160, 1, 2)])
def test_rows_of_no_lse_add_nothing(n_q, n_kv, m, value):
    """A row whose lse is -inf adds nothing, whatever its query holds."""
    hd, n = 64, 300
    c = ref.make_cache(m, [(m, n), (1, 40)], n_kv, hd, 16)
    x = queries(m, m + 1, n_q, hd)
    _, lse, _, _ = ref.attention(c, x, hd ** -0.5)
    lse = lse.float()
    masked = [0, m // 2, m - 1]
    lse[masked] = -math.inf
    lse[1, n_q - 1] = -math.inf                     # one head of a token that counts otherwise
    mass = torch.rand(2, n_kv, c.cap)
    want, tol = ref.attention_mass(c, x, lse, hd ** -0.5, mass)
    x[masked] = value
    x[1, n_q - 1] = value
    got = q.attention_mass(handle(c), x.cuda(), c.q_start.cuda(), lse.cuda(), max_q=m, mass=mass.cuda())
    close(got[0, :, :n], want[0, :, :n], tol[0, :, :n], "mass")
    close(got[1, :, :40], want[1, :, :40], tol[1, :, :40], "mass of the other sequence")
    assert q.device_status() == 0
