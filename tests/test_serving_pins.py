"""Pins of the serving-step definitions (oracle/serving.py) against worked
examples, library routines and invariants, and the argument checks of the
entry points (nothing is launched: no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import serving
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bd.load()


# ----------------------------------------------------------------------------
# e4m3 and the cache


def test_e4m3_table_by_hand_and_against_torch():
    t = serving.e4m3_table()
    for code, value in {0x00: 0.0, 0x01: 2.0 ** -9, 0x07: 7 * 2.0 ** -9, 0x08: 2.0 ** -6,
                        0x38: 1.0, 0x39: 1.125, 0x7e: 448.0, 0xb8: -1.0}.items():
        assert t[code] == value
    lib_values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, lib_values)


def test_e4m3_rounding_against_torch():
    g = torch.Generator().manual_seed(3)
    x = torch.cat([torch.randn(4000, generator=g) * 100, torch.randn(4000, generator=g) * 0.01,
                   torch.tensor([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 447.9, 432.0, 0.0, -0.0])])
    x = x.clamp(-448, 448)
    got = serving.e4m3_encode(x.numpy())
    np.testing.assert_array_equal(got, x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert serving.e4m3_encode(np.array([np.inf, -np.inf, np.nan])).tolist() == [0x7e, 0xfe, 0x7f]
    t = serving.e4m3_table()
    fin = np.arange(256)[np.isfinite(t)]
    np.testing.assert_array_equal(serving.e4m3_encode(t[fin]), fin)


def test_group_scale_by_hand():
    assert serving.group_scale([448.0]) == 1.0
    assert serving.group_scale([448.5, -1.0]) == 2.0
    assert serving.group_scale([-224.0]) == 0.5
    assert serving.group_scale([0.0]) == 2.0 ** -64
    assert serving.group_scale([np.nan, np.inf, 3.5]) == 2.0 ** -7


def test_append_worked_example():
    """A head of d = 1, groups of 4.  Prefix 3 rows (values 1, 2, 4 at scale 1);
    the new row 896 needs the scale 2: the old codes halve in value."""
    codes = serving.e4m3_encode(np.array([1.0, 2.0, 4.0, 7.0, 9.0]).reshape(1, 1, 5, 1))
    c, s = serving.append_q8(codes, np.ones((1, 1, 2)), [3], np.array([896.0, 3.0]).reshape(1, 1, 2, 1), [2], 4)
    assert s.tolist() == [[[2.0, 2.0 ** -7]]]
    assert serving.e4m3_decode(c).ravel().tolist() == [0.5, 1.0, 2.0, 448.0, 384.0]
    assert serving.values(c, s, 4).ravel().tolist() == [1.0, 2.0, 4.0, 896.0, 3.0]
    # the draft row replaced by a small one: the scale shrinks back, the prefix is exact
    c, s = serving.append_q8(c, s, [3], np.array([0.5, 0.0]).reshape(1, 1, 2, 1), [1], 4)
    assert s[0, 0, 0] == 2.0 ** -6
    assert serving.values(c, s, 4).ravel()[:4].tolist() == [1.0, 2.0, 4.0, 0.5]


def test_decode_matches_the_attention_oracle():
    """Over values that bf16 holds, the definition is oracle.decode's."""
    rng = np.random.default_rng(5)
    q = torch.randn((2, 4, 3, 32), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    codes = rng.integers(0, 127, (2, 2, 2, 40, 32)).astype(np.uint8)
    codes[..., ::2] |= 128
    scale = 2.0 ** rng.integers(-9, -5, (2, 2, 2, 3))
    k, v = (serving.values(codes[t], scale[t], 16) for t in (0, 1))
    lens = np.array([0, 35], dtype=np.int32)
    for mode in (0, 1, 2):
        o, l, _, _ = serving.decode(q.double().numpy(), k, v, lens, mode)
        ro, rl = oracle.decode(q, torch.tensor(k).to(torch.bfloat16), torch.tensor(v).to(torch.bfloat16),
                               torch.tensor(lens), mode, 1 / math.sqrt(32))
        np.testing.assert_allclose(o, ro.reshape(o.shape), atol=1e-12)
        np.testing.assert_allclose(l, rl.reshape(l.shape), atol=1e-12)


# ----------------------------------------------------------------------------
# rotary positions


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_relative_and_orthogonal(interleaved):
    rng = np.random.default_rng(7)
    f, _ = serving.rope_freqs(16, 10000.0)
    q, k = rng.standard_normal((2, 1, 1, 1, 24))

    def at(x, p, **kw):
        return serving.rope(x, [[p]], f, interleaved, **kw)
    a = (at(q, 9) * at(k, 4)).sum()
    b = (at(q, 1005) * at(k, 1000)).sum()
    assert abs(a - b) < 1e-10                             # scores depend on the distance
    np.testing.assert_allclose(at(at(q, 77), 77, adjoint=True), q, atol=1e-12)
    np.testing.assert_array_equal(at(q, 0), q)
    np.testing.assert_array_equal(at(q, 5)[..., 16:], q[..., 16:])
    # <m R x, y> = <x, adjoint y>
    y = rng.standard_normal(q.shape)
    assert abs((at(q, 5, mscale=1.3) * y).sum() - (q * at(y, 5, mscale=1.3, adjoint=True)).sum()) < 1e-12


def test_rope_quarter_turn_by_hand():
    x = np.arange(1.0, 5.0).reshape(1, 1, 1, 4)
    f = [np.pi / 2, np.pi]
    np.testing.assert_allclose(serving.rope(x, [[1]], f), [[[[-3, -2, 1, -4]]]], atol=1e-14)
    np.testing.assert_allclose(serving.rope(x, [[1]], f, interleaved=True), [[[[-2, 1, -3, -4]]]], atol=1e-14)


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, trained_len=4096)])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rope_table_matches_the_formula(lib, rot, kw):
    f, m = bd.rope_table(rot, 10000.0, device="cpu", **kw)
    rf, rm = serving.rope_freqs(rot, 10000.0, **kw)
    np.testing.assert_allclose(f.numpy(), rf, rtol=1e-13)
    assert abs(m - rm) < 1e-6
    if kw.get("scaling") == "yarn" and rot == 128:
        assert f[0] == 1.0 and abs(f[-1].item() * 16 - 10000.0 ** (-126 / 128)) < 1e-15


# ----------------------------------------------------------------------------
# verification


def test_verify_keeps_the_target_distribution():
    """Integrated over u and r, the first emitted token has the target's
    distribution, whatever the draft's."""
    p = np.array([[0.5, 0.2, 0.3], [1.0, 0, 0]])
    q = np.array([[0.2, 0.7, 0.1]])
    n = 200
    grid = (np.arange(n) + 0.5) / n
    got = np.zeros(3)
    for x in range(3):
        for u in grid:
            a, t = serving.verify_one([x], q, p, [u], 0.5)
            if a:
                got[x] += q[0, x] / n
            else:
                for r in grid:
                    got[serving.verify_one([x], q, p, [u], r)[1]] += q[0, x] / n / n
    np.testing.assert_allclose(got, p[0], atol=2 / n)


def test_verify_edges_by_hand():
    p = np.array([[0.25, 0.75, 0.0], [0.0, 0.5, 0.5], [0.1, 0.2, 0.7]])
    assert serving.verify_one([1, 2], None, p, [0.7, 0.4], 0.25) == (2, 1)  # all accepted, from row 2
    assert serving.verify_one([1, 2], None, p, [0.75, 0.4], 0.0) == (0, 0)  # 0.75 < 0.75 is false
    assert serving.verify_one([1, 0], None, p, [0.5, 0.0], 0.5) == (1, 2)   # p = 0 refuses at u = 0; ties go up
    assert serving.verify_one([], None, p, [], 0.3) == (0, 1)              # nothing drafted: from row 0
    # nothing left of p - q: from p
    assert serving.verify_one([1], p[:1], p[:2], [np.nan], 0.1) == (0, 0)
    assert serving.draw_from(np.array([0.0, np.nan, -1.0]), 0.5) == -1


# ----------------------------------------------------------------------------
# refusals (host only)

A = 1 << 20  # a 16-byte-aligned fake address; never dereferenced
I, U = bd.BD_ERR_INVALID_ARG, bd.BD_ERR_UNSUPPORTED


def _call(fn, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(**a)


ROPE = dict(q=A, k=A + 4096, q_out=A + 8192, k_out=A + 12288, inv_freq=A, start=None, positions=None, B=2, Hq=4,
            Hkv=2, N=8, d=64, rot_dim=32, period=8, interleaved=0, mscale=1.0, adjoint=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), I), (dict(k=None), I), (dict(k_out=None), I), (dict(inv_freq=None), I),
    (dict(inv_freq=A + 4), I), (dict(q=A + 8), I), (dict(start=A, positions=A), I), (dict(start=A + 2), I),
    (dict(B=0), I), (dict(N=0), I), (dict(period=0), I), (dict(Hkv=0), I), (dict(rot_dim=0), I),
    (dict(rot_dim=80), I), (dict(mscale=float("nan")), I), (dict(interleaved=2), I), (dict(adjoint=-1), I),
    (dict(q_out=A + 4096), I), (dict(k_out=A + 8192), I), (dict(k=None, k_out=None), I),
    (dict(rot_dim=24), U), (dict(d=96, rot_dim=32), U),
])
def test_rope_rejects(lib, kw, status):
    assert _call(bd.bd_rope, ROPE, kw) == status


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(base=1.0), dict(base=float("inf")), dict(scaling=4),
    dict(scaling=1, factor=0.5), dict(scaling=2, rot_dim=2), dict(scaling=3, trained_len=0),
    dict(scaling=3, beta_slow=32.0), dict(mscale=None), dict(inv_freq=None),
])
def test_rope_table_rejects(lib, kw):
    buf, m = (ctypes.c_double * 64)(), ctypes.c_float()
    base = dict(inv_freq=ctypes.addressof(buf), mscale=ctypes.addressof(m), rot_dim=64, base=10000.0, scaling=0,
                factor=2.0, trained_len=4096, beta_fast=32.0, beta_slow=1.0)
    assert _call(bd.bd_rope_table, base, {}) == bd.BD_OK
    assert _call(bd.bd_rope_table, base, kw) == I


APPEND = dict(k_cache=A, v_cache=A + 65536, k_scale=A + 4, v_scale=A + 512, cache_len=A, k_new=A, v_new=A, n_new=None,
              B=2, Hkv=2, b=4, d=64, S_cap=64, group=32, advance=1, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(k_cache=None), I), (dict(v_scale=None), I), (dict(cache_len=None), I), (dict(k_new=None), I),
    (dict(v_new=None), I), (dict(k_new=None, v_new=None, advance=0), I), (dict(k_cache=A + 8), I),
    (dict(k_scale=A + 2), I), (dict(k_new=A + 8), I), (dict(n_new=A + 1), I), (dict(v_cache=A), I),
    (dict(v_scale=A + 4), I), (dict(b=0), I), (dict(B=-1), I), (dict(advance=2), I), (dict(group=0), I),
    (dict(group=48), U), (dict(group=256), U), (dict(d=80), U), (dict(B=65536), U), (dict(Hkv=32768), U),
])
def test_append_q8_rejects(lib, kw, status):
    assert _call(bd.bd_cache_append_q8, APPEND, kw) == status


READ = dict(k_cache=A, v_cache=A + 65536, k_scale=A + 4, v_scale=A + 512, cache_len=A, k_out=A + (1 << 18),
            v_out=A + (1 << 19), B=2, Hkv=2, d=64, S_cap=64, group=32, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(k_out=None), I), (dict(v_out=A + (1 << 18)), I), (dict(k_out=A), I), (dict(v_out=A + 8), I),
    (dict(S_cap=0), I), (dict(group=20), U), (dict(d=48), U),
])
def test_read_q8_rejects(lib, kw, status):
    assert _call(bd.bd_cache_read_q8, READ, kw) == status


DECODE = dict(q_blk=A, k_cache=A, v_cache=A + 65536, k_scale=A + 4, v_scale=A + 512, cache_len=A, out=A, lse=A, B=2,
              Hq=4, Hkv=2, b=8, d=64, intra_block_mode=0, stream=None, S_cap=64, group=32, workspace=A,
              workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(k_scale=None), I), (dict(v_scale=A + 6), I), (dict(q_blk=A + 8), I), (dict(Hq=3), I), (dict(S_cap=4), I),
    (dict(intra_block_mode=3), I), (dict(workspace_bytes=16), I), (dict(workspace=A + 16), I), (dict(group=-1), I),
    (dict(v_cache=A), I), (dict(group=8), U), (dict(d=256), U), (dict(B=40000, Hkv=2, Hq=2), U),
])
def test_decode_q8_rejects(lib, kw, status):
    assert _call(bd.bd_attn_decode_q8, DECODE, kw) == status


VERIFY = dict(draft=A, draft_prob=A, target_prob=A, u_accept=A, u_sample=A, n_draft=None, n_accept=A, next_token=A + 64,
              B=2, b=4, V=100, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(draft=None), I), (dict(target_prob=None), I), (dict(u_accept=None), I), (dict(u_sample=None), I),
    (dict(n_accept=None), I), (dict(next_token=A), I), (dict(draft_prob=A + 2), I), (dict(n_draft=A + 3), I),
    (dict(B=0), I), (dict(b=0), I), (dict(V=0), I), (dict(V=4194305), U),
])
def test_verify_rejects(lib, kw, status):
    assert _call(bd.bd_spec_verify, VERIFY, kw) == status


def test_tensor_checks_refuse_cpu_tensors():
    """The tensor calls name the argument that is not on a GPU."""
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 1, 32, 64), dtype=torch.float8_e4m3fn)
    s = torch.ones((1, 1, 1))
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        bd.rope(q, None, torch.ones(16, dtype=torch.float64))
    with pytest.raises(ValueError, match="k_cache must be"):
        bd.cache_append_q8(c, c, s, s, n, q[:, :1], q[:, :1], 32)
    with pytest.raises(ValueError, match="group must be"):
        bd.decode_q8(q, c, c, s, s, n, 0, 33)
    with pytest.raises(ValueError, match="draft must be"):
        bd.spec_verify(n[None], None, torch.zeros(1, 2, 8), torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(ValueError, match="scaling"):
        bd.rope_table(64, scaling="other", device="cpu")
