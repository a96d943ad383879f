"""GPU parity of the serving step over a KV cache in 8 bits (rotary positions,
quantised append and read back, decode, verification) with the fp64 / integer
definitions of oracle/serving.py, alone and in a run of them together.

Tolerances.  Codes, scales, counts and tokens are exact.  bf16 outputs round
by at most 2^-8 of the value.  Rotary positions: cosine, sine and the turn's
fraction in fp32 add at most 2^-20 mscale (|x_a| + |x_b|).  Decode: a score is
off by at most e = scale (qk 2^-23 (d + 8) + 2^-17 sqrt(d) amax terms), with qk
= max_j sum |q k|: products are exact, sums of d terms lose at most a step
each, and the queries' two 8-bit halves hold a value to 2^-17 of the row's
largest; probabilities round by at most 2^-11 (halves) and 2^-21 (exponential),
so out is off by 2^-8 |out| + (e + 2^-11 + 2^-21) (sum p |v| + |out|), and lse
by e + 2^-20 (1 + |lse|) + n 2^-24 for a sum of n terms.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serving
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bd.load()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def bits(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def ok():
    torch.cuda.synchronize()
    assert bd.device_status() == bd.BD_OK


# ----------------------------------------------------------------------------
# rotary positions


def check_rope(y, x, pos, f, inter, m, adj):
    ref = serving.rope(f64(x), pos, f, inter, m, adj)
    half = len(f)
    mag = np.zeros(ref.shape)
    a = slice(0, 2 * half, 2) if inter else slice(0, half)
    b = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    mag[..., a] = mag[..., b] = np.abs(f64(x)[..., a]) + np.abs(f64(x)[..., b])
    err = np.abs(f64(y) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * m * mag).all(), err.max()
    # dims behind the turned ones are copied
    assert torch.equal(y[..., 2 * half:].cpu(), x[..., 2 * half:])


@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot,period", [
    (2, 4, 2, 33, 128, 128, 33), (1, 1, 1, 1, 64, 64, 1), (3, 6, 2, 130, 64, 32, 65),
    (2, 3, 3, 7, 32, 16, 7), (1, 32, 8, 64, 128, 48, 32), (5, 2, 1, 257, 32, 32, 100),
])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_matches_the_definition(B, Hq, Hkv, N, d, rot, period, inter):
    g = gen(N + d)
    q, k = randn(g, B, Hq, N, d), randn(g, B, Hkv, N, d)
    f, m = bd.rope_table(rot, scaling="yarn", factor=4.0, trained_len=128)
    start = torch.randint(0, 2 ** 30, (B,), generator=g).to(torch.int32)
    pos = start[:, None].long() + torch.arange(N) % period
    for adj in (False, True):
        qo, ko = bd.rope(q.cuda(), k.cuda(), f, start=start.cuda(), period=period,
                         interleaved=inter, mscale=m, adjoint=adj)
        ok()
        check_rope(qo, q, pos.numpy(), f64(f), inter, m, adj)
        check_rope(ko, k, pos.numpy(), f64(f), inter, m, adj)


def test_rope_given_positions_queries_alone_and_in_place():
    g = gen(9)
    q = randn(g, 2, 3, 20, 64)
    pos = torch.randint(-1000, 2 ** 31 - 1, (2, 20), generator=g).to(torch.int32)
    f, _ = bd.rope_table(48)
    x = q.cuda()
    out, none = bd.rope(x, None, f, positions=pos.cuda(), q_out=x)
    ok()
    assert none is None and out.data_ptr() == x.data_ptr()
    check_rope(x, q, pos.numpy(), f64(f), False, 1.0, False)


def test_rope_same_positions_in_both_halves_of_the_training_form():
    g = gen(10)
    L = 40
    x = randn(g, 1, 2, L, 128)
    q = torch.cat([x, x], 2).cuda()
    f, _ = bd.rope_table(128)
    qo, _ = bd.rope(q, None, f, period=L)
    ok()
    assert torch.equal(qo[:, :, :L], qo[:, :, L:])
    assert torch.equal(qo[:, :, 0], q[:, :, 0])  # position 0 does not turn


def test_rope_gradient_by_differences():
    """The map is linear: <rope(x + e) - rope(x), y> = <e, adjoint(y)>."""
    g = gen(11)
    f, m = bd.rope_table(64, scaling="yarn", factor=8.0, trained_len=64)
    x, y = randn(g, 1, 2, 50, 64), randn(g, 1, 2, 50, 64)
    dx, _ = bd.rope(y.cuda(), None, f, mscale=m, adjoint=True)
    a, _ = bd.rope(x.cuda(), None, f, mscale=m)
    ok()
    for b, h, n, e in ((0, 0, 3, 5), (0, 1, 49, 40), (0, 1, 0, 63)):
        z = x.clone()
        z[b, h, n, e] += 2.0
        step = float(z[b, h, n, e]) - float(x[b, h, n, e])
        zo, _ = bd.rope(z.cuda(), None, f, mscale=m)
        diff = ((f64(zo) - f64(a)) * f64(y)).sum() / step
        # two outputs differ, each of the two values rounded by 2^-8
        tol = 2.0 ** -8 * ((np.abs(f64(zo)) + np.abs(f64(a)))[b, h, n] * np.abs(f64(y))[b, h, n]).sum() / step
        assert abs(diff - float(dx[b, h, n, e])) <= tol + 2.0 ** -8 * abs(float(dx[b, h, n, e]))


# ----------------------------------------------------------------------------
# quantised append and read back


def make_cache(B, H, S, d, group, seed, spread=3):
    """Codes and power-of-two scales with whatever was left behind: NaN codes
    and wild scales behind the lengths are the caller's to add."""
    g = gen(seed)
    codes = torch.randint(0, 256, (B, H, S, d), generator=g, dtype=torch.uint8)
    codes = torch.where((codes & 127) == 127, codes & 0x80, codes)
    scale = torch.exp2(torch.randint(-8 - spread, -8 + spread, (B, H, -(-S // group)), generator=g).float())
    return codes, scale


def cuda_cache(codes):
    return codes.cuda().view(torch.float8_e4m3fn)


@pytest.mark.parametrize("d", [128, 64, 32])
@pytest.mark.parametrize("group", [16, 32, 64, 128])
def test_append_matches_the_definition(d, group):
    B, H, b, S = 7, 2, 70, 333
    lens = [0, 1, group, group + 5, S - b, S - 3, 200]
    counts = [b, 3, 0, b, b, 3, 1]
    g = gen(d + group)
    kc, ks = make_cache(B, H, S, d, group, 1)
    vc, vs = make_cache(B, H, S, d, group, 2)
    kn, vn = randn(g, B, H, b, d, scale=3.0), randn(g, B, H, b, d)
    kn[0, 0, 5] = 0                      # rows and groups of zeros
    kn[1, 1, :3] = 0
    vn[3, 0, 0, 0] = 3.0e38              # the largest scale
    vn[3, 1, 1] = vn[3, 1, 1] * 1e-30    # below the smallest
    kn[4, 0, 2, 1], kn[4, 0, 2, 2], kn[4, 0, 3, 0] = float("inf"), float("-inf"), float("nan")
    dev = [cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda()]
    cl = i32(lens).cuda()
    bd.cache_append_q8(*dev, cl, kn.cuda(), vn.cuda(), group, n_new=i32(counts).cuda(), advance=False)
    ok()
    assert cl.tolist() == lens
    for codes, scale, new, c, s in ((kc, ks, kn, dev[0], dev[2]), (vc, vs, vn, dev[1], dev[3])):
        rc, rs = serving.append_q8(codes.numpy(), scale.numpy(), lens, f64(new), counts, group)
        got = bits(c)
        same = (got == rc) | (((got & 127) == 127) & ((rc & 127) == 127))  # a NaN's sign is free
        assert same.all(), np.argwhere(~same)[:5]
        np.testing.assert_array_equal(f64(s), rs)


def test_append_whole_blocks_advances_and_repeats():
    """n_new = None; the same draft written twice changes nothing; advancing
    leaves the rows; lengths alone advance without rows."""
    B, H, b, d, group, S = 3, 2, 24, 64, 32, 128
    lens = [0, 17, 100]
    g = gen(3)
    kc, ks = make_cache(B, H, S, d, group, 4)
    vc, vs = make_cache(B, H, S, d, group, 5)
    kn, vn = randn(g, B, H, b, d).cuda(), randn(g, B, H, b, d).cuda()
    dev = [cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda()]
    cl = i32(lens).cuda()
    bd.cache_append_q8(*dev, cl, kn, vn, group, advance=False)
    once = [t.clone() for t in dev]
    bd.cache_append_q8(*dev, cl, kn, vn, group)
    ok()
    for a, c in zip(once, dev):
        np.testing.assert_array_equal(bits(a), bits(c))
    assert cl.tolist() == [24, 41, 124]
    bd.cache_append_q8(*dev, cl, None, None, group, n_new=i32([1, 0, 4]).cuda())
    ok()
    assert cl.tolist() == [25, 41, 128]


@pytest.mark.parametrize("lens,counts", [([5, -1], [4, 4]), ([5, 40], [4, 9]), ([5, 0], [4, 11]), ([5, 3], [4, -2])])
def test_append_out_of_range_leaves_the_sequence(lens, counts):
    B, H, b, d, group, S = 2, 1, 10, 32, 16, 48
    kc, ks = make_cache(B, H, S, d, group, 6)
    kn = randn(gen(6), B, H, b, d).cuda()
    dev = [cuda_cache(kc), cuda_cache(kc), ks.cuda(), ks.cuda()]
    cl = i32(lens).cuda()
    bd.cache_append_q8(*dev, cl, kn, kn, group, n_new=i32(counts).cuda())
    torch.cuda.synchronize()
    assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT
    assert bd.device_status() == bd.BD_OK
    assert cl.tolist() == [9, lens[1]]
    np.testing.assert_array_equal(bits(dev[0])[1], kc.numpy()[1])
    np.testing.assert_array_equal(f64(dev[2])[1], ks.numpy()[1])


@pytest.mark.parametrize("d,group,S", [(128, 64, 200), (64, 16, 77), (32, 128, 300)])
def test_read_back_matches_the_definition(d, group, S):
    B, H = 4, 3
    lens = [0, 1, S, S // 2]
    kc, ks = make_cache(B, H, S, d, group, 7)
    vc, vs = make_cache(B, H, S, d, group, 8)
    vs = vs * 1.37  # a scale that is no power of two rounds
    ko = torch.full((B, H, S, d), 7.0, dtype=torch.bfloat16).cuda()
    vo = ko.clone()
    bd.cache_read_q8(cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), group, k_out=ko, v_out=vo)
    ok()
    rk, rv = serving.values(kc.numpy(), ks.numpy(), group), serving.values(vc.numpy(), vs.numpy(), group)
    for i, n in enumerate(lens):
        np.testing.assert_array_equal(f64(ko)[i, :, :n], rk[i, :, :n])
        # the product rounds to fp32, then to bf16
        assert (np.abs(f64(vo)[i, :, :n] - rv[i, :, :n]) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(rv[i, :, :n])).all()
        assert (ko[i, :, n:] == 7).all() and (vo[i, :, n:] == 7).all()


def test_read_back_bad_length_is_reported():
    kc, ks = make_cache(2, 1, 32, 32, 16, 9)
    ko, vo = bd.cache_read_q8(cuda_cache(kc), cuda_cache(kc), ks.cuda(), ks.cuda(), i32([33, 32]).cuda(), 16)
    torch.cuda.synchronize()
    assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT
    assert (ko[0] == 0).all()
    np.testing.assert_array_equal(f64(ko)[1], serving.values(kc.numpy(), ks.numpy(), 16)[1])


# ----------------------------------------------------------------------------
# decode


def check_decode(out, lse, q, k, v, lens, mode):
    d = q.shape[-1]
    ro, rl, mag, qk = serving.decode(f64(q), k, v, lens, mode)
    o, l = f64(out), f64(lse)
    empty = rl == -np.inf
    assert (o[empty] == 0).all() and (l[empty] == -np.inf).all()
    amax = np.abs(f64(q)).max(-1)
    kmax = np.abs(np.nan_to_num(k)).max()
    e = (qk * 2.0 ** -23 * (d + 8) + 2.0 ** -17 * math.sqrt(d) * amax * kmax) / math.sqrt(d)
    tol = 2.0 ** -8 * np.abs(ro) + (e + 2.0 ** -11 + 2.0 ** -21)[..., None] * (mag + np.abs(ro)) + 1e-30
    err = np.abs(o - ro)
    assert (err <= tol)[~empty].all(), (err[~empty] / tol[~empty]).max()
    n = k.shape[2]
    lt = e + 2.0 ** -20 * (1 + np.abs(rl)) + n * 2.0 ** -24
    err = np.abs(l[~empty] - rl[~empty])
    assert (err <= lt[~empty]).all(), err.max()


def decode_case(B, Hq, H, b, d, S, group, lens, mode, seed):
    g = gen(seed)
    q = randn(g, B, Hq, b, d)
    kv = []
    for t in (0, 1):
        x = torch.randn((B, H, S, d), generator=g) * torch.exp2(torch.randint(-2, 3, (B, H, 1, 1), generator=g).float())
        codes, scale = serving.append_q8(np.zeros((B, H, S, d), np.uint8), np.ones((B, H, -(-S // group))),
                                         [0] * B, f64(x.to(torch.bfloat16)), [S] * B, group)
        # whatever earlier sequences left behind the visible rows: NaN codes
        # and, in groups with no visible row, scales that are no scales
        for i in range(B):
            n = int(lens[i]) + (b if mode != 2 else 0)
            codes[i, :, n:] = 0x7f
            scale[i, :, -(-n // group):] = (0.0, float("nan"))[t]
        kv.append((torch.tensor(codes), torch.tensor(scale, dtype=torch.float32)))
    return q, kv


def run_decode(q, kv, lens, mode, group, **kw):
    (kc, ks), (vc, vs) = kv
    out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), mode, group, **kw)
    ok()
    k, v = (serving.values(c.numpy(), s.numpy(), group) for c, s in kv)
    check_decode(out, lse, q, k, v, lens, mode)
    return out, lse


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("d,group", [(128, 64), (128, 16), (64, 128), (32, 32)])
def test_decode_matches_the_definition(d, group, mode):
    b = 28
    lens = [0, 1, 99, 100, 101, 128, 300]
    q, kv = decode_case(len(lens), 8, 2, b, d, 340, group, lens, mode, d + group + mode)
    run_decode(q, kv, lens, mode, group)


@pytest.mark.parametrize("Hq,H,b", [(1, 1, 1), (8, 1, 1), (4, 4, 3), (6, 2, 1), (8, 2, 33), (16, 2, 64), (5, 1, 130)])
def test_decode_head_groups_and_block_sizes(Hq, H, b):
    """One row to several 128-row tiles of a unit, whole groups and odd ones."""
    for mode in (0, 1):
        lens = [40, 257]
        q, kv = decode_case(2, Hq, H, b, 64, 400, 32, lens, mode, 10 * Hq + b)
        run_decode(q, kv, lens, mode, 32)


@pytest.mark.parametrize("d,group", [(128, 64), (128, 16), (64, 128), (64, 32), (32, 16), (32, 128)])
@pytest.mark.parametrize("Hq,H,b", [(4, 1, 1), (4, 2, 4), (3, 1, 3), (3, 1, 5), (4, 2, 8), (4, 1, 5), (8, 2, 8), (1, 1, 31)])
def test_decode_few_rows(Hq, H, b, d, group):
    """Up to 8, 16 and 32 query rows a unit, over prefixes that end inside
    and at the end of a step, a part of one and a run of 16 keys."""
    for mode in (0, 1, 2):
        lens = [1, 33, 128, 255, 1100, 0 if mode == 2 else 64]
        q, kv = decode_case(len(lens), Hq, H, b, d, 1200, group, lens, mode, 100 * Hq + 10 * b + d + mode)
        run_decode(q, kv, lens, mode, group)


@pytest.mark.parametrize("rows", [(4, 1, 1), (8, 2, 7)])
@pytest.mark.parametrize("grid", [1, 2, 5, 31])
def test_decode_few_rows_split_over_any_grid(grid, rows):
    Hq, H, b = rows
    lens = [2500, 3, 700, 0, 129, 1]
    q, kv = decode_case(6, Hq, H, b, 128, 2600, 64, lens, 1, grid)
    assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
    try:
        run_decode(q, kv, lens, 1, 64)
    finally:
        bd.bd_attn_debug_set_grid(0)


@pytest.mark.parametrize("grid", [1, 3, 5, 37])
def test_decode_split_over_any_grid(grid):
    lens = [1500, 3, 700, 0, 129]
    q, kv = decode_case(5, 4, 2, 16, 128, 1600, 64, lens, 1, grid)
    assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
    try:
        run_decode(q, kv, lens, 1, 64)
    finally:
        bd.bd_attn_debug_set_grid(0)


def test_decode_rows_of_different_size_and_sharp_scores():
    """Query rows from 0 to 2^20, one dim far above the rest; scores that leave
    one key all the mass."""
    lens = [500]
    q, kv = decode_case(1, 4, 1, 8, 128, 520, 64, lens, 1, 77)
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 2.0 ** -20
    q[0, 0, 2] *= 64
    q[0, 1, 3, 5] = 200.0
    q[0, 2, 4] *= 2.0 ** -100
    run_decode(q, kv, lens, 1, 64)


def test_decode_groups_of_very_different_scale():
    """Value groups 2^40 apart, and groups of zeros at the smallest scale that
    hold most of the mass."""
    lens = [256]
    q, kv = decode_case(1, 4, 1, 4, 64, 300, 32, lens, 0, 78)
    (kc, ks), (vc, vs) = kv
    vs[0, 0, 1] *= 2.0 ** 20
    vs[0, 0, 2] *= 2.0 ** -20
    vc[0, 0, 96:160] = 0
    vs[0, 0, 3:5] = 2.0 ** -64
    q *= 2
    run_decode(q, [(kc, ks), (vc, vs)], lens, 0, 32)


def test_decode_few_rows_sharp_scores_and_scales():
    """One row per head: rows of different size, value groups 2^40 apart, a
    group of zeros, scales that are no powers of two."""
    lens = [700]
    q, kv = decode_case(1, 8, 2, 1, 128, 800, 32, lens, 1, 85)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -20
    q[0, 2] *= 64
    q[0, 3, 0, 5] = 200.0
    q[0, 4] *= 2.0 ** -100
    run_decode(q, kv, lens, 1, 32)
    (kc, ks), (vc, vs) = kv
    vs[0, :, 1] *= 2.0 ** 20
    vs[0, :, 2] *= 2.0 ** -20
    vc[0, :, 96:160] = 0
    vs[0, :, 3:5] = 2.0 ** -64
    ks = ks * (0.7 + torch.rand(ks.shape, generator=gen(86)))
    run_decode(q, [(kc, ks), (vc, vs)], lens, 1, 32)


def test_decode_any_positive_scale():
    lens = [200, 77]
    q, kv = decode_case(2, 4, 2, 5, 128, 220, 16, lens, 0, 79)
    g = gen(80)
    kv = [(c, s * (0.7 + torch.rand(s.shape, generator=g))) for c, s in kv]
    run_decode(q, kv, lens, 0, 16)


def test_decode_not_a_number():
    """NaN and infinite query rows give NaN rows, a NaN key NaN in the rows
    that see it; every other row is untouched."""
    lens = [100]
    q, kv = decode_case(1, 2, 2, 4, 64, 128, 16, lens, 1, 81)
    q[0, 0, 1, 3], q[0, 0, 2, 0] = float("nan"), float("inf")
    kv[0][0][0, 1, 102, 7] = 0x7f  # seen by the block's rows 2 and 3 of kv-head 1
    (kc, ks), (vc, vs) = kv
    out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 1, 16)
    ok()
    nan = torch.isnan(lse).cpu()
    want = torch.zeros((1, 2, 4), dtype=torch.bool)
    want[0, 0, 1] = want[0, 0, 2] = want[0, 1, 2] = want[0, 1, 3] = True
    assert torch.equal(nan, want)
    assert torch.equal(torch.isnan(out).all(-1).cpu(), want) and torch.equal(torch.isnan(out).any(-1).cpu(), want)


@pytest.mark.parametrize("b", [1, 40])
@pytest.mark.parametrize("grid", [1, 7])
def test_decode_not_a_number_in_a_cut_unit(b, grid):
    """The same where a unit's pieces are merged, and for few rows."""
    lens = [1000]
    q, kv = decode_case(1, 2, 1, b, 128, 1100, 16, lens, 0, 84)
    q[0, 0, 0, 9] = float("-inf")
    (kc, ks), (vc, vs) = kv
    assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
    try:
        out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 0, 16)
        ok()
        want = torch.zeros((1, 2, b), dtype=torch.bool)
        want[0, 0, 0] = True
        assert torch.equal(torch.isnan(lse).cpu(), want) and torch.equal(torch.isnan(out).any(-1).cpu(), want)
        kc[0, 0, 700, 3] = 0x7f  # a key that every row sees
        out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 0, 16)
        ok()
        assert torch.isnan(lse).all() and torch.isnan(out).all()
    finally:
        bd.bd_attn_debug_set_grid(0)


def test_decode_bad_length_is_reported():
    lens = [30, 60, 20]
    q, kv = decode_case(3, 2, 1, 4, 64, 64, 16, [30, 20, 20], 0, 82)
    (kc, ks), (vc, vs) = kv
    for bad in (61, -1):
        cl = i32([30, bad, 20]).cuda()
        out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), cl, 0, 16)
        torch.cuda.synchronize()
        assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT
        assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).all()
        assert torch.isfinite(lse[0]).all() and torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("S", [200, 1536, 1537])
@pytest.mark.parametrize("b", [1, 40, 140])
def test_decode_rows_without_a_key(b, S):
    """Empty prefixes and invalid lengths beside good ones, in caches whose
    units are never cut and in one where they may be."""
    lens = [150, 0, 33, 0]
    q, kv = decode_case(4, 4, 2, b, 64, S, 32, lens, 2, 90 + b)
    run_decode(q, kv, lens, 2, 32)
    (kc, ks), (vc, vs) = kv
    good, lse_good = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 2, 32)
    out, lse = bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32([150, S + 1, 33, -1]).cuda(), 2, 32)
    torch.cuda.synchronize()
    assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT
    for i in (1, 3):
        assert torch.isnan(lse[i]).all() and torch.isnan(out[i]).all()
    for i in (0, 2):
        assert torch.equal(out[i], good[i]) and torch.equal(lse[i], lse_good[i])


def test_decode_wait_that_runs_out_is_reported():
    """One K tile never arrives: the bounded wait runs out, the launch reports
    it, the next one is right."""
    lens = [900, 300]
    q, kv = decode_case(2, 4, 1, 20, 128, 1000, 64, lens, 0, 89)
    (kc, ks), (vc, vs) = kv
    assert bd.bd_attn_debug_inject_fault(1) == bd.BD_OK
    bd.decode_q8(q.cuda(), cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 0, 64)
    torch.cuda.synchronize()
    assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT
    run_decode(q, kv, lens, 0, 64)


def test_decode_is_deterministic_and_takes_a_workspace_and_a_stream():
    lens = [900, 5, 260]
    q, kv = decode_case(3, 8, 2, 20, 128, 1000, 128, lens, 1, 83)
    a = run_decode(q, kv, lens, 1, 128)
    ws = torch.empty(bd.workspace_bytes(3, 8, 2, 20, 128, 1000), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_decode(q, kv, lens, 1, 128, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def off16(shape, dtype=torch.bfloat16):
    """A contiguous buffer on a 16-byte boundary that is none of 32 bytes."""
    n = math.prod(shape)
    t = torch.zeros(n + 16, dtype=dtype, device="cuda")[8:8 + n].view(shape)
    assert t.data_ptr() % 32 == 16 and t.is_contiguous()
    return t


@pytest.mark.parametrize("b", [1, 40])
def test_buffers_on_16_byte_boundaries(b):
    """New rows, read-back rows, queries and outputs where a 32-byte access
    would be misaligned; whole units and cut ones."""
    lens = [600, 40]
    q, kv = decode_case(2, 4, 2, b, 128, 700, 32, lens, 0, 87)
    (kc, ks), (vc, vs) = kv
    k, v = (serving.values(c.numpy(), s.numpy(), 32) for c, s in kv)
    for grid in (0, 3):
        assert bd.bd_attn_debug_set_grid(grid) == bd.BD_OK
        try:
            qd, out = off16(q.shape), off16(q.shape)
            qd.copy_(q)
            _, lse = bd.decode_q8(qd, cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 0, 32, out=out)
            ok()
            check_decode(out, lse, q, k, v, lens, 0)
        finally:
            bd.bd_attn_debug_set_grid(0)
    ko, vo = off16(k.shape), off16(k.shape)
    bd.cache_read_q8(cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda(), i32(lens).cuda(), 32, k_out=ko, v_out=vo)
    new = off16((2, 2, b, 128))
    new.copy_(randn(gen(88), 2, 2, b, 128))
    dev = [cuda_cache(kc), cuda_cache(vc), ks.cuda(), vs.cuda()]
    bd.cache_append_q8(*dev, i32(lens).cuda(), new, new, 32)
    ok()
    for i, n in enumerate(lens):
        np.testing.assert_array_equal(f64(ko)[i, :, :n], k[i, :, :n])
        np.testing.assert_array_equal(f64(vo)[i, :, :n], v[i, :, :n])
    rc, rs = serving.append_q8(kc.numpy(), ks.numpy(), lens, f64(new), [b, b], 32)
    for i, n in enumerate(lens):
        np.testing.assert_array_equal(bits(dev[0])[i, :, :n + b], rc[i, :, :n + b])


# ----------------------------------------------------------------------------
# verification


def verify_case(B, b, V, seed, point=False, n_draft=None):
    g = gen(seed)
    z = torch.randn((B, b + 1, V), generator=g)
    p = torch.softmax(2 * z + 0.8 * torch.randn((B, b + 1, V), generator=g), -1)
    q = torch.softmax(2 * z[:, :b], -1)
    x = q.argmax(-1) if point else torch.multinomial(q.reshape(B * b, V), 1, generator=g).reshape(B, b)
    u, r = torch.rand((B, b), generator=g), torch.rand((B,), generator=g)
    return x.to(torch.int32), None if point else q, p, u, r, n_draft


def run_verify(x, q, p, u, r, nd):
    n, t = bd.spec_verify(x.cuda(), None if q is None else q.cuda(), p.cuda(), u.cuda(), r.cuda(),
                          n_draft=None if nd is None else i32(nd).cuda())
    ok()
    for i in range(x.shape[0]):
        m = x.shape[1] if nd is None else nd[i]
        want = serving.verify_one(x[i, :m].tolist(), None if q is None else q[i].double().numpy(), p[i].double().numpy(),
                                  u[i].double().numpy(), float(r[i]))
        assert (int(n[i]), int(t[i])) == want, i


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 1024, 1025, 8192, 50001])
@pytest.mark.parametrize("point", [False, True])
def test_verify_matches_the_definition(V, point):
    run_verify(*verify_case(9, 5, V, V, point))


def test_verify_long_drafts_and_draft_counts():
    run_verify(*verify_case(6, 70, 300, 1, n_draft=[0, 1, 32, 33, 70, 64]))
    x, q, p, u, r, _ = verify_case(4, 40, 200, 2)
    run_verify(x, q, p, torch.zeros_like(u), r, None)   # everything accepted: the bonus row


def test_verify_edges():
    x, q, p, u, r, _ = verify_case(8, 3, 40, 3)
    p[0, 0] = q[0, 0]                       # p - q leaves nothing: drawn from p
    u[0, 0] = float("nan")                  # never accepted
    p[1, 0, int(x[1, 0])] = 0.0             # a token that the target never takes, at u = 0
    u[1, 0] = 0.0
    r[2] = 0.0
    r[3] = 1.0 - 2.0 ** -24                 # the two ends of the draw
    p[4, 0, 5] = float("nan")
    u[4, 0] = 2.0                           # refused: NaN weights count as 0
    u[5] = 0.0
    p[5] = 0.0
    p[5, :, 7] = 1.0                        # one token has all the mass
    x[5] = 7
    u[6, 0] = 1.0
    q[6, 0, int(x[6, 0])] = p[6, 0, int(x[6, 0])]  # u q = p is a refusal
    run_verify(x, q, p, u, r, None)
    p[7, 0] = 0.0
    q[7, 0] = 0.0
    run_verify(x, q, p, u, r, None)         # no mass at all: -1


def test_verify_bad_tokens_and_counts_are_reported():
    x, q, p, u, r, _ = verify_case(4, 3, 50, 4)
    x[1, 2] = 50
    x[2, 0] = -1
    n, t = bd.spec_verify(x.cuda(), q.cuda(), p.cuda(), u.cuda(), r.cuda(), n_draft=i32([3, 3, 3, 4]).cuda())
    torch.cuda.synchronize()
    assert bd.device_status() == bd.BD_ERR_DEVICE_TIMEOUT
    assert n[1:].tolist() == [0, 0, 0] and t[1:].tolist() == [-1, -1, -1] and int(t[0]) >= 0
    # a bad token behind the drafted ones is not looked at
    run_verify(x, q, p, u, r, [3, 2, 0, 3])


# ----------------------------------------------------------------------------
# together


def step(bufs, group, f):
    """One step of a serving loop: rotate the block, write it as a draft,
    attend to it both ways, verify, keep the accepted rows."""
    q, k, v, kc, vc, ks, vs, cl, x, dp, tp, u, r, out = bufs
    qr, kr = bd.rope(q, k, f, start=cl)
    bd.cache_append_q8(kc, vc, ks, vs, cl, kr, v, group, advance=False)
    o0, l0 = bd.decode_q8(qr, kc, vc, ks, vs, cl, 0, group)
    o1, l1 = bd.decode_q8(qr, kc, vc, ks, vs, cl, 1, group)
    n, t = bd.spec_verify(x, dp, tp, u, r)
    bd.cache_append_q8(kc, vc, ks, vs, cl, None, None, group, n_new=n)
    for dst, src in zip(out, (qr, kr, o0, l0, o1, l1, n, t)):
        dst.copy_(src)


@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_loop_step_by_step(captured):
    """Three steps over one growing cache, checked against the definitions at
    each; the same steps replayed from a captured graph."""
    B, Hq, H, b, d, S, group, V = 3, 8, 2, 12, 64, 200, 32, 500
    g = gen(12)
    f, _ = bd.rope_table(64)
    codes = [np.zeros((B, H, S, d), np.uint8) for _ in (0, 1)]
    scales = [np.ones((B, H, -(-S // group))) for _ in (0, 1)]
    lens = np.array([0, 31, 150])
    pre = [f64(randn(g, B, H, 150, d)) for _ in (0, 1)]
    for t in (0, 1):
        codes[t], scales[t] = serving.append_q8(codes[t], scales[t], [0] * B, pre[t], lens, group)
    kc, vc = (cuda_cache(torch.tensor(c)) for c in codes)
    ks, vs = (torch.tensor(s, dtype=torch.float32).cuda() for s in scales)
    cl = i32(lens.tolist()).cuda()
    new = lambda *shape, dt=torch.bfloat16: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    out = (new(B, Hq, b, d), new(B, H, b, d), new(B, Hq, b, d), new(B, Hq, b, dt=torch.float32), new(B, Hq, b, d),
           new(B, Hq, b, dt=torch.float32), new(B, dt=torch.int32), new(B, dt=torch.int32))
    bufs = [new(B, Hq, b, d), new(B, H, b, d), new(B, H, b, d), kc, vc, ks, vs, cl, new(B, b, dt=torch.int32),
            new(B, b, V, dt=torch.float32), new(B, b + 1, V, dt=torch.float32), new(B, b, dt=torch.float32),
            new(B, dt=torch.float32), out]
    graph = None
    if captured:
        keep = [t.clone() for t in (kc, vc, ks, vs, cl)]
        for t in bufs[:3] + bufs[8:13]:
            t.zero_()
        step(bufs, group, f)  # first calls outside the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(bufs, group, f)
        for dst, src in zip((kc, vc, ks, vs, cl), keep):
            dst.copy_(src)
        ok()
    for it in range(3):
        q, k, v = randn(g, B, Hq, b, d), randn(g, B, H, b, d), randn(g, B, H, b, d)
        x, dp, tp, u, r, _ = verify_case(B, b, V, 50 + it)
        for dst, src in zip(bufs, (q, k, v)):
            dst.copy_(src)
        for dst, src in zip(bufs[8:13], (x, dp, tp, u, r)):
            dst.copy_(src)
        if captured:
            graph.replay()
        else:
            step(bufs, group, f)
        ok()
        qr, kr, o0, l0, o1, l1, n, t = out
        pos = lens[:, None] + np.arange(b)
        check_rope(qr, q, pos, f64(f), False, 1.0, False)
        check_rope(kr, k, pos, f64(f), False, 1.0, False)
        for s, rows in ((0, f64(kr)), (1, f64(v))):
            codes[s], scales[s] = serving.append_q8(codes[s], scales[s], lens, rows, [b] * B, group)
        np.testing.assert_array_equal(bits(kc), codes[0])
        np.testing.assert_array_equal(bits(vc), codes[1])
        kv = [serving.values(c, s, group) for c, s in zip(codes, scales)]
        check_decode(o0, l0, qr, *kv, lens, 0)
        check_decode(o1, l1, qr, *kv, lens, 1)
        for i in range(B):
            want = serving.verify_one(x[i].tolist(), dp[i].double().numpy(), tp[i].double().numpy(),
                                      u[i].double().numpy(), float(r[i]))
            assert (int(n[i]), int(t[i])) == want
        lens = lens + f64(n).astype(np.int64)
        assert cl.tolist() == lens.tolist()


def test_rope_around_the_training_form():
    """rope, fwd, bwd and the rotation's adjoint: the gradient of q and k
    before the rotation, against fp64."""
    from oracle import backward
    B, Hq, H, L, b, d = 1, 2, 1, 64, 16, 128
    g = gen(13)
    q, k, v, do = (randn(g, B, h, 2 * L, d) for h in (Hq, H, H, Hq))
    f, m = bd.rope_table(128, scaling="linear", factor=2.0)
    qr, kr = bd.rope(q.cuda(), k.cuda(), f, period=L)
    out, lse = bd.fwd(qr, kr, v.cuda(), L, b)
    dqr, dkr, dv = bd.bwd(qr, kr, v.cuda(), out, lse, do.cuda(), L, b)
    dq, dk = bd.rope(dqr, dkr, f, period=L, adjoint=True)
    ok()
    pos = np.tile(np.arange(2 * L) % L, (B, 1))
    rq, rk, _ = backward.fwd_bwd(qr.cpu(), kr.cpu(), v, do, L, b, 1 / math.sqrt(d))
    for got, ref in ((dq, rq), (dk, rk)):
        ref = serving.rope(ref.reshape(got.shape), pos, f64(f), adjoint=True)
        # the backward's own bound, 2^-5 of the largest, which the rotation
        # stretches by at most sqrt(2)
        assert np.abs(f64(got) - ref).max() <= 1.5 * 2.0 ** -5 * np.abs(ref).max()
