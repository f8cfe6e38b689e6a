"""GPU: the serving calls at the borders of their kernels: alignments, runs that
end inside a row group, long caches, rounding, and no bounded wait that gives up.
The checks and their bounds are test_gpu_serving's."""
import numpy as np
import pytest

import w8_quantized_linear_b200 as bn
from oracle import serving as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

from test_gpu_parity import dev, host  # noqa: E402
from test_gpu_serving import Attend  # noqa: E402


@pytest.fixture(autouse=True)
def _no_wait_timeouts():
    bn.device_wait_timeout(reset=True)
    yield
    torch.cuda.synchronize()
    assert bn.device_wait_timeout(reset=True) == 0


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("B,L,H,Hkv,P", [
    (65, 4, 32, 8, 130),    # 5 row groups a head (the last of 16 rows), two token tiles each
    (128, 2, 64, 8, 100),   # one token tile a row group: a group begins as the one before ends
    (33, 4, 32, 8, 1290)])  # runs of 6: from one row group into the next at any tile
def test_prefix_attention_of_many_row_groups(B, L, H, Hkv, P, mode):
    """Several row groups a CTA, each of one or a few token tiles: what a group's
    last product leaves is complete before it is read, call after call."""
    a = Attend(B, L, H, Hkv, P, 3, [i % 4 for i in range(B)])
    first = bn.prefix_attention(mode, *a.d)
    a.check(mode, first)
    for _ in range(50):
        got = bn.prefix_attention(mode, *a.d)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
