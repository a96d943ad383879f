"""GPU: attention and cache calls on a stream that is not the current one, while
the current one is busy: outputs and scratch that a call makes neither wait for
the current stream's queue nor lie in memory that the queue is still using."""
import pytest
import torch

import bd_inputs
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build

pytestmark = pytest.mark.gpu


def test_outputs_and_scratch_on_the_stream_of_the_call():
    build.build()
    bd.load()
    L, b, d = 128, 16, 128
    q, k, v = (t.cuda() for t in bd_inputs.fwd_inputs(1, 4, 2, L, d, seed=5))
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    out, lse = bd.fwd(q, k, v, L, b)
    qb, kc, vc, cl = (t.cuda() for t in bd_inputs.decode_inputs(2, 8, 2, 28, d, 300, cache_len=[100, 200], seed=1))
    conf = torch.rand((2, 300), generator=torch.Generator().manual_seed(7)).cuda()
    mod = torch.ones((2, 300), dtype=torch.uint8, device="cuda")
    tokens = torch.zeros((2, 8), dtype=torch.int32, device="cuda")

    def calls(stream):
        got = [*bd.fwd(q, k, v, L, b, stream=stream), *bd.bwd(q, k, v, out, lse, do, L, b, stream=stream),
               *bd.decode(qb, kc, vc, cl, 0, stream=stream), bd.spec_accept(tokens, tokens, stream=stream)]
        # (rows behind a prefix's kept ones are scratch)
        _, _, _, n, score = bd.sprint_prune(kc, vc, cl, conf, mod, want_score=True, stream=stream)
        return got + [n, score]

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sizes = want + [torch.empty(bd.bd_attn_bwd_workspace_bytes(1, 4, L) // 4, device="cuda"),
                    torch.empty(bd.bd_sprint_workspace_bytes(2, 300) // 4, device="cuda")]
    used = [torch.full_like(t, 3) for t in sizes for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms of the current stream
    copies = [t.clone() for t in used]
    del used  # free for the current stream, whose copies are still to come
    got = calls(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in copies)
    for a, c in zip(got, want):
        assert torch.equal(a, c)
    assert bd.device_status() == bd.BD_OK
