"""GPU: the forms of the serving step over a cache in 8 bits that batches, long
vocabularies and the training form take, against oracle/serving.py; helpers and
tolerances are tests/test_gpu_serving.py's."""
import pytest
import torch

from oracle import serving
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build
from test_gpu_serving import (check_decode, check_rope, cuda_cache, decode_case, f64, gen, i32, ok, randn, run_decode,
                              run_verify, verify_case)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bd.load()
    assert torch.cuda.is_available()


# ----------------------------------------------------------------------------
# rotary positions: sizes that give a CTA several heads


def heads_per_cta(B, Hq, Hkv, N, d):
    """The launch's rule: as many as leave 8 CTAs to each of 148 SMs."""
    tiles = B * -(-N // (256 // (d // 16)))
    groups = min(Hq + Hkv, max(1, -(-8 * 148 // tiles)))
    return -(-(Hq + Hkv) // groups)


@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot,period,inter,heads", [
    (2, 23, 7, 4099, 128, 128, 4099, False, 6),   # keys begin inside a CTA, and inside its 4 loads
    (4, 32, 8, 4096, 128, 64, 2048, True, 14),    # both halves of the training form
    (6, 8, 2, 4099, 64, 32, 5000, True, 3),
    (1, 9, 4, 70001, 32, 16, 70001, False, 5),
    (1, 13, 0, 70001, 32, 32, 35001, False, 5),   # queries alone
])
def test_rope_several_heads_to_a_cta(B, Hq, Hkv, N, d, rot, period, inter, heads):
    assert heads_per_cta(B, Hq, Hkv, N, d) == heads
    g = gen(N + d)
    q = randn(g, B, Hq, N, d)
    k = randn(g, B, Hkv, N, d) if Hkv else None
    f, m = bd.rope_table(rot, scaling="yarn", factor=4.0, trained_len=128)
    start = torch.randint(0, 2 ** 20, (B,), generator=g).to(torch.int32)
    rows = sorted({0, 1, N - 1, N - 2, *torch.randint(0, N, (60,), generator=g).tolist()})
    pos = (start[:, None].long() + torch.arange(N) % period)[:, rows].numpy()
    for adj, place in ((False, False), (True, True)):
        qd, kd = q.cuda(), None if k is None else k.cuda()
        qo, ko = bd.rope(qd, kd, f, start=start.cuda(), period=period, interleaved=inter, mscale=m, adjoint=adj,
                         q_out=qd if place else None, k_out=kd if place else None)
        ok()
        check_rope(qo[:, :, rows], q[:, :, rows], pos, f64(f), inter, m, adj)
        if k is not None:
            check_rope(ko[:, :, rows], k[:, :, rows], pos, f64(f), inter, m, adj)
        if not adj:
            whole = qo
    # every row: turning back gives the rows again, off by two roundings of 2^-8
    # of a pair's length, which the turn keeps
    back, _ = bd.rope(whole, None, f, start=start.cuda(), period=period, interleaved=inter, mscale=1 / m, adjoint=True)
    ok()
    x = q.cuda().float()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    length = (a * a + b * b).sqrt() * (1 + 2.0 ** -6)
    y = back.float() - x
    ya, yb = (y[..., :rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    tol = length * (3 * 2.0 ** -8)
    assert (ya.abs() <= tol).all() and (yb.abs() <= tol).all() and (y[..., rot:] == 0).all()


# ----------------------------------------------------------------------------
# decode: more sequences than a warp has lanes


@pytest.mark.parametrize("Hq,H,b", [(4, 1, 1), (8, 2, 7), (4, 1, 40)])
@pytest.mark.parametrize("B", [33, 70])
@pytest.mark.parametrize("grid", [0, 3, 40])
def test_decode_more_sequences_than_lanes(B, Hq, H, b, grid):
    """The work list's second and third round of lengths: zeros, single keys
    and long prefixes in every round, whole units and cut ones."""
    g = gen(B + b)
    lens = torch.randint(0, 260, (B,), generator=g).tolist()
    lens[::7] = [0] * len(lens[::7])
    lens[3], lens[31], lens[32], lens[B - 1] = 900, 1, 640, 700
    q, kv = decode_case(B, Hq, H, b, 64, 960, 32, lens, 0, B + b)
    assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
    try:
        for mode in (1, 2):
            run_decode(q, kv, lens, mode, 32)
    finally:
        bd.bd_attn_debug_set_grid(0)


def test_decode_more_sequences_than_lanes_with_bad_lengths():
    """Sequences of an invalid length beside good ones in every round."""
    B, S = 70, 300
    lens = [(37 * i) % 250 for i in range(B)]
    bad = [i for i in range(B) if i % 9 == 4]
    for Hq, H, b in ((4, 1, 1), (4, 1, 40)):
        q, kv = decode_case(B, Hq, H, b, 64, S, 32, lens, 0, 7)
        (kc, ks), (vc, vs) = kv
        dev = (cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda())
        wrong = [(-1, S + 1)[i % 2] if i in bad else n for i, n in enumerate(lens)]
        out, lse = bd.decode_q8(q.cuda(), *dev, i32(wrong).cuda(), 0, 32)
        torch.cuda.synchronize()
        assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT
        good = [i for i in range(B) if i not in bad]
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        k, v = (serving.values(c.numpy()[good], t.numpy()[good], 32) for c, t in kv)
        check_decode(out[good], lse[good], q[good], k, v, [lens[i] for i in good], 0)


# ----------------------------------------------------------------------------
# decode on the 128-row tiles: scales and NaN as on the kernel for few rows


@pytest.mark.parametrize("d,group", [(128, 32), (64, 16), (32, 64)])
def test_decode_tiles_value_groups_far_apart_and_any_scale(d, group):
    lens = [700]
    q, kv = decode_case(1, 8, 2, 16, d, 800, group, lens, 1, 91)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -20
    q[0, 2] *= 64
    q[0, 3, 0, 5] = 200.0
    q[0, 4] *= 2.0 ** -100
    run_decode(q, kv, lens, 1, group)
    (kc, ks), (vc, vs) = kv
    vs[0, :, 1] *= 2.0 ** 20
    vs[0, :, 2] *= 2.0 ** -20
    vc[0, :, 3 * group:5 * group] = 0
    vs[0, :, 3:5] = 2.0 ** -64
    ks = ks * (0.7 + torch.rand(ks.shape, generator=gen(92)))
    run_decode(q, [(kc, ks), (vc, vs)], lens, 1, group)
    vs = vs * (0.7 + torch.rand(vs.shape, generator=gen(93)))
    run_decode(q, [(kc, ks), (vc, vs)], lens, 1, group)


@pytest.mark.parametrize("grid", [0, 1, 5])
def test_decode_tiles_not_a_number(grid):
    """40 rows a head: NaN and infinite rows give NaN rows, a NaN key NaN in
    the rows that see it; every other row is untouched."""
    b, lens = 40, [600]
    q, kv = decode_case(1, 2, 2, b, 64, 700, 16, lens, 1, 81)
    q[0, 0, 1, 3], q[0, 0, 22, 0] = float("nan"), float("inf")
    kv[0][0][0, 1, 602, 7] = 0x7f  # seen by the block's rows from 2 on of kv-head 1
    (kc, ks), (vc, vs) = kv
    assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
    try:
        out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 1, 16)
        ok()
    finally:
        bd.bd_attn_debug_set_grid(0)
    want = torch.zeros((1, 2, b), dtype=torch.bool)
    want[0, 0, 1] = want[0, 0, 22] = True
    want[0, 1, 2:] = True
    assert torch.equal(torch.isnan(lse).cpu(), want)
    assert torch.equal(torch.isnan(out).all(-1).cpu(), want) and torch.equal(torch.isnan(out).any(-1).cpu(), want)


# ----------------------------------------------------------------------------
# verification


@pytest.mark.parametrize("B,b,V", [(37, 3, 1001), (38, 3, 1000), (40, 2, 4096), (64, 1, 50001)])
@pytest.mark.parametrize("point", [False, True])
def test_verify_batches(B, b, V, point):
    """Both kernels (the one with smaller CTAs from 38 sequences on)."""
    run_verify(*verify_case(B, b, V, B + V, point))


@pytest.mark.parametrize("V", [131072, 131073, 300001, 4194304])
@pytest.mark.parametrize("point", [False, True])
def test_verify_long_vocabularies(V, point):
    """More segments to a CTA than a warp has lanes; draws from both ends, the
    middle and the last entries."""
    g = gen(V)
    p = torch.rand((1, 2, V), generator=g)
    q = torch.rand((1, 1, V), generator=g)
    p[0, :, :V // 3] = 0  # the first CTAs have no mass
    p[0, 0, V // 3:] += 1e-3
    p, q = p / p.sum(-1, keepdim=True), q / q.sum(-1, keepdim=True)
    x = i32([[5]])
    for u, r in ((1.0, 0.0), (1.0, 0.3), (1.0, 0.7), (1.0, 1.0 - 2.0 ** -24), (0.0, 0.999)):
        # refused (p(x) = 0), and nothing drafted: from the row itself
        for nd in (None, [0]):
            run_verify(x, None if point else q, p, torch.full((1, 1), u), torch.full((1,), r), nd)


# ----------------------------------------------------------------------------
# calls at once, and again


@pytest.mark.parametrize("b", [1, 40])
def test_decode_on_two_streams_at_once(b):
    """Calls that overlap, each with a workspace of its own, give what they
    give alone, bit for bit, call after call."""
    cases = []
    for seed in (1, 2):
        lens = [1500, 40, 700 + seed]
        q, kv = decode_case(3, 8, 2, b, 128, 1600, 64, lens, 0, seed)
        (kc, ks), (vc, vs) = kv
        args = (q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 0, 64)
        ws = torch.empty(bd.workspace_bytes(3, 8, 2, b, 128, 1600), dtype=torch.uint8, device="cuda")
        cases.append((args, ws, bd.decode_q8(*args), torch.cuda.Stream()))
    ok()
    for _ in range(10):
        got = []
        for args, ws, _, s in cases:
            with torch.cuda.stream(s):
                got.append([bd.decode_q8(*args, workspace=ws) for _ in range(3)])
        ok()
        for (_, _, want, _), outs in zip(cases, got):
            for out, lse in outs:
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_verify_repeats_itself():
    x, q, p, u, r, _ = verify_case(40, 4, 30000, 9)
    args = [t.cuda() for t in (x, q, p, u, r)]
    first = bd.spec_verify(*args)
    for _ in range(10):
        again = bd.spec_verify(*args)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    ok()


def test_outputs_made_on_the_stream_of_the_call():
    """A call on a stream that is not the current one, which is busy: its
    outputs neither wait for the current stream's queue (zeros among them) nor
    lie in memory that the queue is still using."""
    lens = [100, 60]
    q, kv = decode_case(2, 8, 2, 3, 64, 128, 32, lens, 0, 5)
    (kc, ks), (vc, vs) = kv
    dev = (cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda())
    q = q.cuda()
    f, _ = bd.rope_table(64)
    x, dp, tp, u, r = (t.cuda() for t in verify_case(2, 3, 90, 1)[:5])

    def calls(stream):
        return [*bd.rope(q, None, f, stream=stream)[:1], *bd.cache_read_q8(*dev, 32, stream=stream),
                *bd.decode_q8(q, *dev, 0, 32, stream=stream), *bd.spec_verify(x, dp, tp, u, r, stream=stream)]

    want = [t.clone() for t in calls(None)]
    ok()
    side = torch.cuda.Stream()
    used = [torch.full_like(t, 3) for t in want for _ in range(4)]
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
    ok()
