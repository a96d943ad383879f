"""GPU: the serving step over a cache in 8 bits at the edges of what its header
allows, against oracle/serving.py; helpers and tolerances are
tests/test_gpu_serving.py's."""
import numpy as np
import pytest
import torch

from oracle import serving
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build
from test_gpu_serving import bits, cuda_cache, decode_case, f64, gen, i32, ok, randn, run_decode, verify_case

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


# ----------------------------------------------------------------------------
# the cache


@pytest.mark.parametrize("d,group", [(128, 64), (32, 16)])
def test_append_and_read_back_of_the_largest_values(d, group):
    """The largest bf16, infinities and NaN: finite values read back finite,
    and stay when rows join their group."""
    B, H, S, b = 1, 2, 2 * group, 9
    g = gen(d)
    new = randn(g, B, H, b, d)
    top = torch.finfo(torch.bfloat16).max
    new[0, :, 2, ::3], new[0, :, 3, 1::3] = top, -top
    new[0, 0, 4, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    dev = [torch.zeros((B, H, S, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in (0, 1)]
    dev += [torch.ones((B, H, S // group), device="cuda") for _ in (0, 1)]
    cl = i32([0]).cuda()
    rc, rs = np.zeros((B, H, S, d), np.uint8), np.ones((B, H, S // group))
    for lens, rows in (([0], new), ([b], randn(g, B, H, 3, d))):
        bd.cache_append_q8(*dev, cl, rows.cuda(), rows.cuda(), group)
        ok()
        rc, rs = serving.append_q8(rc, rs, lens, f64(rows), [rows.shape[2]], group)
        for c, s in ((dev[0], dev[2]), (dev[1], dev[3])):
            got = bits(c)
            assert ((got == rc) | (((got & 127) == 127) & ((rc & 127) == 127))).all()
            np.testing.assert_array_equal(f64(s), rs)
        ko, vo = bd.cache_read_q8(*dev, cl, group)
        ok()
        want = serving.values(rc, rs, group)
        for o in (ko, vo):
            np.testing.assert_array_equal(f64(o)[:, :, :int(cl[0])], want[:, :, :int(cl[0])])
            assert torch.isfinite(o[0, :, 2:4]).all() and torch.isnan(o).sum() == 1


@pytest.mark.parametrize("d,group", [(128, 64), (64, 16), (32, 128)])
def test_append_rounds_kept_values_below_the_normal_codes(d, group):
    """Every code kept at scale 1, a row that asks for 2 to 2^11, then a small
    one in its place: kept values are exact from 2^-6 of the scale on, and what
    is rounded below stays so."""
    B, H, S = 1, 2, 2 * group
    n = group - 2
    kc = torch.arange(n * d).reshape(1, 1, n, d) % 256
    kc = torch.where((kc & 127) == 127, 9, kc).to(torch.uint8).expand(B, H, n, d)
    codes = torch.zeros((B, H, S, d), dtype=torch.uint8)
    codes[:, :, :n] = kc
    for k in (1, 2, 5, 11):
        dev = [codes.cuda().view(torch.float8_e4m3fn) for _ in (0, 1)]
        dev += [torch.ones((B, H, S // group), device="cuda") for _ in (0, 1)]
        cl = i32([n]).cuda()
        rc, rs = codes.numpy(), np.ones((B, H, S // group))
        for top in (448.0 * 2.0 ** k, 0.5):
            row = torch.full((B, H, 1, d), top, dtype=torch.bfloat16)
            bd.cache_append_q8(*dev, cl, row.cuda(), row.cuda(), group, advance=False)
            ok()
            rc, rs = serving.append_q8(rc, rs, [n], f64(row), [1], group)
            for c, s in ((dev[0], dev[2]), (dev[1], dev[3])):
                np.testing.assert_array_equal(bits(c)[:, :, :n + 1], rc[:, :, :n + 1])
                np.testing.assert_array_equal(f64(s), rs)
        was, now = (serving.values(x, y, group)[:, :, :n] for x, y in ((codes.numpy(), np.ones_like(rs)), (rc, rs)))
        large = np.abs(was) >= 2.0 ** (k - 6)
        assert (was[large] == now[large]).all() and (was != now).any()


# ----------------------------------------------------------------------------
# decode

# (B, Hq, Hkv, b): 4 and 28 rows a unit on the kernel for few rows (28 below d =
# 128 alone), 80 on the 128-row tiles
ROWS = [(4, 1, 1), (8, 2, 7), (4, 2, 40)]


def far_scales(g, H, S, d, group, lo, hi):
    """A cache of one sequence: random keys, value codes between 1 and 448 in
    size, and V scales of any power of two from 2^lo to 2^hi."""
    kc = torch.randint(0x30, 0x48, (1, H, S, d), generator=g).to(torch.uint8)
    vc = torch.randint(0x38, 0x7f, (1, H, S, d), generator=g).to(torch.uint8)
    kc, vc = ((c | (torch.randint(0, 2, c.shape, generator=g) * 128).to(torch.uint8)) for c in (kc, vc))
    n = -(-S // group)
    return (kc, torch.ones(1, H, n)), (vc, torch.exp2(torch.randint(lo, hi + 1, (1, H, n), generator=g).float()))


@pytest.mark.parametrize("Hq,H,b", ROWS)
@pytest.mark.parametrize("scales", [(-100, 30), (30, -100), (-64, 90), (120, -80), (-100, -100), (120, 120)])
def test_decode_two_keys_whose_value_scales_lie_far_apart(Hq, H, b, scales):
    """Equal scores: half the weight each, whatever their V scales; the two in
    one tile, and in tiles of different warps and warpgroups.  (A scale's
    logarithm is off by 2^-22 of it, 120 at most, and counts in both keys.)"""
    d, group = 64, 32
    for at in (16, 40, 100, 150, 500):
        S, lens = 704, [at + 1]
        vc = torch.full((1, H, S, d), 0x38, dtype=torch.uint8)
        kc = torch.zeros((1, H, S, d), dtype=torch.uint8)
        kc[:, :, 1:at] = 0xfe  # -448: no weight beside 0
        q = torch.ones((1, Hq, b, d), dtype=torch.bfloat16)
        vs = torch.full((1, H, S // group), scales[0], dtype=torch.float32)
        vs[:, :, at // group:] = scales[1]
        kv = (kc, torch.ones(1, H, S // group)), (vc, torch.exp2(vs))
        out, lse = run_decode(q, kv, lens, 2, group)
        assert (lse.cpu() - np.log(2.0)).abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("Hq,H,b", ROWS)
@pytest.mark.parametrize("d,group", [(128, 16), (128, 64), (64, 32), (32, 128)])
@pytest.mark.parametrize("lo,hi,size", [(-64, 20, 1.0), (-100, 110, 1.0), (-100, 110, 30.0), (60, 110, 1.0)])
def test_decode_value_scales_of_any_size(Hq, H, b, d, group, lo, hi, size):
    """Random scales of V, scores close together and far apart, in whole units
    and cut ones."""
    g = gen(d + group + hi)
    lens = [900]
    kv = far_scales(g, H, 1024, d, group, lo, hi)
    q = randn(g, 1, Hq, b, d, scale=size)
    for grid in (0, 3):
        assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
        try:
            run_decode(q, kv, lens, 1, group)
        finally:
            bd.bd_attn_debug_set_grid(0)


@pytest.mark.parametrize("Hq,H,b", ROWS)
@pytest.mark.parametrize("d,qe,ke", [(128, -80, 80), (64, -100, 98), (128, -125, 118), (32, -60, 60)])
def test_decode_small_queries_over_large_keys(Hq, H, b, d, qe, ke):
    """Query rows of 2^qe, keys of 2^ke: scores of order one and more."""
    lens = [300]
    g = gen(d - qe)
    (kc, ks), v = far_scales(g, H, 400, d, 32, -3, 0)
    q = (randn(g, 1, Hq, b, d).float().clamp(-3, 3) * 2.0 ** qe).to(torch.bfloat16)
    q[:, 0] = (q[:, 0].float() * 2.0 ** -4).to(torch.bfloat16) if qe > -120 else q[:, 0]
    run_decode(q, ((kc, ks * 2.0 ** ke), v), lens, 0, 32)


@pytest.mark.parametrize("Hq,H,b", [(4, 1, 1), (2, 1, 20)])
@pytest.mark.parametrize("shift", [0.0, 0.3, 1.0])
def test_decode_one_sharp_key_beside_a_quarter_of_a_million(Hq, H, b, shift):
    """One key with about half the mass, the rest spread evenly over 2^18
    others, whose weights are the smallest that f16 holds beside it: within the
    bound of the header, n 2^-28 448 max p s beside the roundings of each key."""
    d, group, n = 32, 128, 1 << 18
    g = gen(5)
    kc = torch.zeros((1, 1, n + 128, d), dtype=torch.uint8)
    kc[0, 0, 0] = 0x38  # 1
    vc = torch.randint(0x38, 0x7f, (1, 1, n + 128, d), generator=g).to(torch.uint8)
    ks, vs = torch.ones(1, 1, (n + 128) // group), torch.full((1, 1, (n + 128) // group), 2.0 ** -8)
    q = torch.full((1, Hq, b, d), (np.log(float(n)) + shift) / np.sqrt(d), dtype=torch.float32).to(torch.bfloat16)
    lens = [n]
    out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 2, group)
    ok()
    k, v = (serving.values(c.numpy(), s.numpy(), group) for c, s in ((kc, ks), (vc, vs)))
    ro, rl, mag, qk = serving.decode(f64(q), k, v, lens, 2)
    p = np.exp(qk.max() / np.sqrt(d) - rl)  # the sharp key's weight
    assert 0.4 < p.min() and p.max() < 0.8
    # check_decode's bound, with the header's term for weights below f16's range
    e = (qk * 2.0 ** -23 * (d + 8) + 2.0 ** -17 * np.sqrt(d) * np.abs(f64(q)).max(-1)) / np.sqrt(d)
    tol = 2.0 ** -8 * np.abs(ro) + (e + 2.0 ** -11 + 2.0 ** -21)[..., None] * (mag + np.abs(ro))
    tol = tol + (n * 2.0 ** -28 * 448 * 2.0 ** -8 * p)[..., None]
    assert (np.abs(f64(out) - ro) <= tol).all()
    assert (np.abs(f64(lse) - rl) <= e + 2.0 ** -20 * (1 + np.abs(rl)) + n * 2.0 ** -24).all()


@pytest.mark.parametrize("Hq,H,b", ROWS)
@pytest.mark.parametrize("grid", [0, 2, 7])
def test_decode_far_scales_in_some_sequences(Hq, H, b, grid):
    """V scales far apart in every other sequence, a prefix's first or last
    groups alone: a CTA goes from segments of one kind to the other."""
    B, d, group, S = 6, 64, 32, 1100
    lens = [1000, 300, 64, 900, 1, 513]
    q, kv = decode_case(B, Hq, H, b, d, S, group, lens, 1, 17)
    (kc, ks), (vc, vs) = kv
    vc[vc == 0] = 0x38  # (a code of 0 beside far larger values would ask for more than P holds)
    vs[0, :, 0] = 2.0 ** -90
    vs[2, :, :] = torch.exp2(torch.arange(vs.shape[2]).float() * 40 - 64)
    vs[3, :, 20:] *= 2.0 ** 100
    vs[5, 0, 15] = 2.0 ** -100
    for i in range(B):  # no scale behind the visible rows
        vs[i, :, -(-(lens[i] + b) // group):] = float("nan")
    assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
    try:
        run_decode(q, ((kc, ks), (vc, vs)), lens, 1, group)
    finally:
        bd.bd_attn_debug_set_grid(0)


@pytest.mark.parametrize("Hq,H,b", ROWS)
@pytest.mark.parametrize("grid", [0, 3])
def test_decode_not_a_number_beside_far_scales(Hq, H, b, grid):
    """NaN and infinite query rows give NaN rows, a NaN key NaN in the rows
    that see it, no other row changes."""
    g = gen(23)
    lens = [700]
    (kc, ks), (vc, vs) = far_scales(g, H, 900, 64, 32, -100, 100)
    q = randn(g, 1, Hq, b, 64)
    assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
    try:
        def call(q, kc):
            out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 1, 32)
            ok()
            return out.cpu(), lse.cpu()
        good, lse_good = call(q, kc)
        assert torch.isfinite(good).all() and torch.isfinite(lse_good).all()
        q[0, 0, 0, 3], q[0, 1, b - 1, 0] = float("nan"), float("-inf")
        kc = kc.clone()
        kc[0, H - 1, 700 + b // 2, 5] = 0x7f  # seen by the rows from b // 2 on of the last kv-head
        out, lse = call(q, kc)
    finally:
        bd.bd_attn_debug_set_grid(0)
    want = torch.zeros((1, Hq, b), dtype=torch.bool)
    want[0, 0, 0] = want[0, 1, b - 1] = True
    want[0, Hq - Hq // H:, b // 2:] = True
    assert torch.equal(torch.isnan(lse), want)
    assert torch.equal(torch.isnan(out).all(-1), want) and torch.equal(torch.isnan(out).any(-1), want)
    assert torch.equal(out[~want], good[~want]) and torch.equal(lse[~want], lse_good[~want])
