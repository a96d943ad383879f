"""GPU: the serving step over a cache in 8 bits where offsets pass 32 bits: 2^26
positions of 128 values a head, 2^32 rotated values, 2^32 probabilities.  Most
of each buffer is one value, so the answers are known without an oracle's pass."""
import math

import numpy as np
import pytest
import torch

from oracle import serving
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build
from test_gpu_serving import bits, check_rope, f64, gen, i32, ok, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bd.load()
    assert torch.cuda.is_available()
    yield
    torch.cuda.empty_cache()


def test_cache_of_more_than_32_bits():
    """Append, decode and read back at both ends and in the middle of two
    heads of 2^26 positions (2^33 codes each)."""
    B, H, d, group, S = 1, 2, 128, 64, (1 << 26) + 200
    G = -(-S // group)
    g = gen(1)
    # every key -448 (no weight) and every value 1 but where rows are appended
    kc = torch.full((B, H, S, d), 0xfe, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = torch.full((B, H, S, d), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks, vs = torch.ones((B, H, G), device="cuda"), torch.ones((B, H, G), device="cuda")
    cl = i32([0]).cuda()
    at = [5, (1 << 25) + 3, (1 << 26) - 40]
    rows = []
    for p in at:  # three rows each, keys of zeros: the weight of all of them
        v = randn(g, B, H, 3, d)
        cl.fill_(p)
        bd.cache_append_q8(kc, vc, ks, vs, cl, torch.zeros_like(v).cuda(), v.cuda(), group, advance=False)
        ok()
        rows.append(v)
        # as the definition writes them; what was there keeps its value
        lo = p // group * group
        c = np.full((B, H, group * 2, d), 0x38, np.uint8)
        rc, rs = serving.append_q8(c, np.ones((B, H, 2)), [p - lo], f64(v), [3], group)
        n = p - lo + 3
        np.testing.assert_array_equal(bits(vc[:, :, lo:lo + n]), rc[:, :, :n])
        np.testing.assert_array_equal(f64(vs[:, :, lo // group:lo // group + 2]), rs)
        assert (kc[:, :, p:p + 3].view(torch.uint8) == 0).all()
    n = at[-1] + 3
    # rows of the appended keys' groups that follow them are no rows of the cache
    # for append, and hold what they held: still without weight
    scale = [float(vs[0, h, p // group]) for h in range(H) for p in at]
    want = np.stack([np.concatenate([serving.e4m3_decode(bits(vc[0, h, p:p + 3])) * float(vs[0, h, p // group])
                                     for p in at]).mean(0) for h in range(H)])
    assert all(s > 0 for s in scale)
    for b in (1, 10, 40):  # 2, 20 and 80 rows a unit
        q = torch.ones((B, 2 * H, b, d), dtype=torch.bfloat16, device="cuda")
        cl.fill_(n)
        out, lse = bd.decode_q8(q, kc, vc, ks, vs, cl, 2, group)
        ok()
        assert np.abs(f64(lse) - math.log(9.0)).max() <= 2.0 ** -14
        ref = np.repeat(want, 2, axis=0)[None, :, None, :]
        mag = np.abs(want).max() + 4  # 9 weights, each rounded by 2^-11
        assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag).all()
    cl.fill_(n)
    ko, vo = bd.cache_read_q8(kc, vc, ks, vs, cl, group)
    ok()
    for p, v in zip(at, rows):
        assert (ko[:, :, p:p + 3] == 0).all()
        got = serving.e4m3_decode(bits(vc[:, :, p:p + 3])) * f64(vs[:, :, p // group])[..., None, None]
        np.testing.assert_array_equal(f64(vo[:, :, p:p + 3]), got)
    assert (ko[:, :, (1 << 25) + 1000:(1 << 25) + 9000] == -448).all() and (vo[:, :, 1000:9000] == 1).all()
    assert (ko[:, :, n:] == 0).all() and (vo[:, :, n:] == 0).all()


def test_rope_of_more_than_32_bits():
    """2^32 values and more, in place: the last heads' rows."""
    H, N, d = 34, 1 << 20, 128
    f, _ = bd.rope_table(d)
    g = gen(2)
    x = torch.ones((1, H, N, d), dtype=torch.bfloat16, device="cuda")
    idx = [0, 1, 77777, N - 2, N - 1]
    keep = randn(g, 1, 2, len(idx), d)
    x[:, H - 2:, idx] = keep.cuda()
    bd.rope(x, None, f, q_out=x)
    ok()
    pos = np.array([idx])
    check_rope(x[:, H - 2:, idx], keep, pos, f64(f), False, 1.0, False)
    ones = torch.ones((1, 1, len(idx), d), dtype=torch.bfloat16)
    for h in (0, 31):  # (32 and 33 hold `keep`)
        check_rope(x[:, h:h + 1, idx], ones, pos, f64(f), False, 1.0, False)


def test_verify_of_more_than_32_bits():
    """2^32 probabilities and more: the last sequences' rows."""
    B, b, V = 560, 1, 4194304
    p = torch.zeros((B, b + 1, V), device="cuda")
    x = torch.arange(B, dtype=torch.int32)[:, None] * 7000 + 11
    rows = torch.arange(B)
    p[rows, 0, x[:, 0].long()] = 0.5
    p[rows, 0, V - 1 - rows.cuda()] = 0.5
    p[rows, 1, (rows * 3).cuda()] = 1.0
    u = torch.full((B, b), 0.25)
    u[1::2] = 0.75  # refused: what is left of p is its other token
    n, t = bd.spec_verify(x.cuda(), None, p, u.cuda(), torch.full((B,), 0.5).cuda())
    ok()
    assert n.tolist() == [1 - i % 2 for i in range(B)]
    assert t.tolist() == [3 * i if i % 2 == 0 else V - 1 - i for i in range(B)]
