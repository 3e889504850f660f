"""The tile GEMM at chosen tile widths."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk

pytestmark = pytest.mark.gpu

DEV = "cuda"


def done():
    torch.cuda.synchronize()
    assert sk.tile_device_error(clear=True) == 0


@pytest.mark.parametrize("M,N,K", [(4097, 5120, 256), (257, 40000, 272), (1025, 20000, 144), (4100, 5000, 512)])
def test_int8_last_tile_of_a_few_tokens(M, N, K):
    """A pair's last tile holds 1 to 4 tokens: the smallest matrix instruction of 256 rows."""
    rng = np.random.default_rng(M)
    d = lambda a: torch.from_numpy(a).to(DEV)
    q, c = (d(rng.integers(-128, 128, shape, dtype=np.int8)) for shape in ((M, K), (N, K)))
    rs, cs = (d(rng.uniform(0.5, 1.5, n).astype(np.float32) / 1000) for n in (M, N))
    w = sk.WeightInt8(c, cs)
    expected = (q.double() @ c.double().T).float() * rs[:, None] * cs[None]      # the sum is exact: below 2^53
    for ws in (sk.make_int8_workspace(), None):
        assert torch.equal(sk.gemm_int8(q, rs, w, torch.float32, workspace=ws), expected)
        done()
