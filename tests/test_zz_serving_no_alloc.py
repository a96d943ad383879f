"""The serving step over a cache in 8 bits with every buffer the caller's: the
calls allocate no device memory, and can be recorded in a CUDA graph captured in
global mode, where any allocation would fail the capture.  Collected last, as
tests/test_zz_no_alloc.py is."""
import pytest
import torch

import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build
from test_gpu_serving import cuda_cache, gen, i32, make_cache, randn, verify_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b", [1, 12, 40])
def test_a_step_allocates_nothing(b):
    build.build()
    bd.load()
    B, Hq, H, d, S, group, V = 5, 8, 2, 128, 2000, 64, 700
    g = gen(b)
    lens = [0, 1500, 77, 900, 1900]
    (kc, ks), (vc, vs) = make_cache(B, H, S, d, group, 1), make_cache(B, H, S, d, group, 2)
    kc, vc, ks, vs, cl = cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda()
    f, _ = bd.rope_table(d)
    q, k, v = randn(g, B, Hq, b, d).cuda(), randn(g, B, H, b, d).cuda(), randn(g, B, H, b, d).cuda()
    x, dp, tp, u, r, _ = verify_case(B, b, V, 3)
    x, dp, tp, u, r = (t.cuda() for t in (x, dp, tp, u, r))
    qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    lse = torch.empty((B, Hq, b), device="cuda")
    ko, vo = (torch.zeros((B, H, S, d), dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    n, t = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(bd.workspace_bytes(B, Hq, H, b, d, S), dtype=torch.uint8, device="cuda")

    def step():
        bd.rope(q, k, f, start=cl, q_out=qr, k_out=kr)
        bd.cache_append_q8(kc, vc, ks, vs, cl, kr, v, group, advance=False)
        bd.decode_q8(qr, kc, vc, ks, vs, cl, 1, group, out=out, lse=lse, workspace=ws)
        bd.spec_verify(x, dp, tp, u, r, n_accept=n, next_token=t)
        bd.cache_append_q8(kc, vc, ks, vs, cl, None, None, group, n_new=n)
        bd.cache_read_q8(kc, vc, ks, vs, cl, group, k_out=ko, v_out=vo)

    keep = [a.clone() for a in (kc, vc, ks, vs, cl)]

    def reset():
        for a, c in zip((kc, vc, ks, vs, cl), keep):
            a.copy_(c)

    step()  # modules load, attributes are set
    torch.cuda.synchronize()
    want = [a.clone() for a in (out, lse, n, t, cl, ko, vo)]
    torch.cuda.synchronize()
    free, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    reset()
    step()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free and torch.cuda.memory_allocated() == held
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="global"):
        step()
    for _ in range(2):
        reset()
        for a in (out, lse):
            a.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip((out, lse, n, t, cl, ko, vo), want):
            assert torch.equal(a, c)
    assert bd.device_status() == bd.BD_OK
