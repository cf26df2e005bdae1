"""The token kernel's bound is one that a kernel with P in a single 16-bit term breaks."""
from __future__ import annotations

import pytest
import torch

from tests import token_ref as ref


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,dtype", [(n, torch.bfloat16) for n in (3, 8, 17, 40, 64)] + [(n, torch.float16) for n in (3, 8, 17)])
def test_one_term_of_p_is_told(n, dtype, d):
    """(With more keys the roundings of one term average out, and the bounds of the sums grow.)"""
    for rows in (8, 16):
        q, k, v = (x.double() for x in ref.make(n, rows, d, dtype, n))
        o, _, tol, _ = ref.attend(q, k, v, dtype, d ** -0.5)
        bad, _, _, _ = ref.attend(q, k, v, dtype, d ** -0.5, once=True)
        assert ((bad - o).abs() > tol).sum() > 20
        # what a last rounding alone does to the definition stays within it
        assert ((o.to(dtype).double() - o).abs() <= tol).all()


def test_the_definition():
    q, k, v = (x.double() for x in ref.make(40, 8, 64, torch.bfloat16, 1))
    o, z, _, _ = ref.attend(q, k, v, torch.bfloat16, 0.2)
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], scale=0.2)[0]
    assert torch.allclose(o, want, atol=1e-13)
    assert torch.allclose(z, torch.logsumexp(q @ k.T * 0.2, 1), atol=1e-13)
