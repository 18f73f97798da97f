"""The 8-bit linear layer where an instance of its kernels is met on purpose:
output edges inside a warp, every kernel that quantizes rows, long sums.
Definitions in 64 bits; what is exact there is compared bit for bit."""
import pytest
import torch

import qlora_bit_frozen_b200 as q
from test_int8_linear import BF, F32, make, rows64, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [17, 40, 64, 90, 129])
@pytest.mark.parametrize("O,I", [(33, 97), (127, 161), (225, 31), (1000, 1025)])
def test_outputs_that_end_inside_a_warp(R, O, I, dtype):
    """Widths off 32, over several runs of eight tokens: every value, and none beside them."""
    W, X, dY, A, B = make(R, O, I, 4, dtype)
    w, nw, s = weight(W)

    def fenced(m):
        buf = torch.full((R * m + 64,), 7.0, dtype=dtype, device="cuda")
        return buf[R * m:], buf[:R * m].view(R, m)

    after, Y = fenced(O)
    q.qlora_linear_fwd(w, X, A, torch.zeros_like(B), 8.0, Y=Y)
    n, sx = rows64(X.float())
    assert torch.equal(Y, (((n @ nw.T).float() * sx[:, None]) * s[None, :]).to(dtype)) and bool((after == 7).all())
    after, dX = fenced(I)
    q.qlora_linear_bwd(w, X, dY, torch.zeros_like(A), B, 8.0, dX=dX)
    n, sg = rows64(dY.float() * s[None, :])
    assert torch.equal(dX, ((n @ nw).float() * sg[:, None]).to(dtype)) and bool((after == 7).all())
