"""GPU: the serving step over a cache in 8 bits at the edges of what its header
allows, against oracle/serving.py; helpers and tolerances are
tests/test_gpu_serving.py's."""
import numpy as np
import pytest
import torch

from oracle import serving
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build
from test_gpu_serving import i32, verify_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bd.load()
    assert torch.cuda.is_available()


# ----------------------------------------------------------------------------
# verification


@pytest.mark.parametrize("B", [6, 40])  # both kernels
@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("out", ["n_accept", "next_token"])
def test_verify_replaces_the_counts_in_place(B, point, out):
    """n_draft's buffer as an output: the counts and tokens of a call with
    buffers of its own, time after time; a bad count among them."""
    b, V = 5, 700
    x, q, p, u, r, _ = verify_case(B, b, V, B, point)
    u = 0.9 + 0.1 * u  # most positions are refused, but the first two of every other sequence
    u[::2, :2] = 0.0
    nd = [5, 3, 0, 1, b + 1, 4] * B
    nd = nd[:B]
    want = []
    for i in range(B):
        m = nd[i]
        want.append((0, -1) if m > b else serving.verify_one(
            x[i, :m].tolist(), None if q is None else q[i].double().numpy(), p[i].double().numpy(),
            u[i].double().numpy(), float(r[i])))
    assert any(0 < n < nd[i] for i, (n, _) in enumerate(want)) and any(n == 0 for n, _ in want)
    args = [x.cuda(), None if q is None else q.cuda(), p.cuda(), u.cuda(), r.cuda()]
    for _ in range(20):
        counts = i32(nd).cuda()
        n, t = bd.spec_verify(*args, n_draft=counts, **{out: counts})
        torch.cuda.synchronize()
        assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT  # the bad count
        assert counts.data_ptr() in (n.data_ptr(), t.data_ptr())
        assert list(zip(n.tolist(), t.tolist())) == want
    assert bd.device_status() == bd.BD_OK
