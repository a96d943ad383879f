"""What the header promises of the serving step over a cache in 8 bits at the
edges of its domain: refusals (host only, nothing is launched) and the
definitions of oracle/serving.py there."""
import numpy as np
import pytest

from oracle import serving
import block_diffusion_lm_attn_b200 as bd
from block_diffusion_lm_attn_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bd.load()


A = 1 << 20  # fake addresses, 64 KB apart and more; never dereferenced
VERIFY = dict(draft=A, draft_prob=2 * A, target_prob=3 * A, u_accept=4 * A, u_sample=5 * A, n_draft=6 * A,
              n_accept=7 * A, next_token=8 * A, B=8, b=4, V=100, stream=None)


@pytest.mark.parametrize("out", ["n_accept", "next_token"])
@pytest.mark.parametrize("at", [A, A + 8 * 4 * 4 - 4, 2 * A, 2 * A + 8 * 4 * 100 * 4 - 4, 3 * A - 28,
                                3 * A + 8 * 5 * 100 * 4 - 4, 4 * A + 64, 5 * A, 6 * A + 4, 6 * A - 4])
def test_verify_refuses_outputs_over_inputs(lib, out, at):
    """The first and last entries of every input, and n_draft's buffer shifted
    by an entry: another sequence's count."""
    assert bd.bd_spec_verify(**{**VERIFY, out: at}) == bd.BD_ERR_INVALID_ARG


@pytest.mark.parametrize("shift", [-28, -4, 0, 4, 28])
def test_verify_refuses_outputs_over_one_another(lib, shift):
    assert bd.bd_spec_verify(**{**VERIFY, "next_token": 7 * A + shift}) == bd.BD_ERR_INVALID_ARG


# ----------------------------------------------------------------------------
# the cache


def test_append_keeps_the_largest_values_finite():
    """255 2^120, the largest bf16, would round to the code of 2^128."""
    big = 255.0 * 2.0 ** 120
    new = np.array([big, -big, 1.0, 248.0 * 2.0 ** 120, np.inf, -np.inf, np.nan]).reshape(1, 1, 7, 1)
    c, s = serving.append_q8(np.zeros((1, 1, 16, 1), np.uint8), np.ones((1, 1, 1)), [0], new, [7], 16)
    assert s[0, 0, 0] == 2.0 ** 120
    v = serving.values(c, s, 16).ravel()[:7] / 2.0 ** 120
    assert v[:6].tolist() == [240.0, -240.0, 0.0, 240.0, 240.0, -240.0] and np.isnan(v[6])
    # kept beside a smaller row, they stay
    c2, s2 = serving.append_q8(c, s, [7], np.ones((1, 1, 1, 1)), [1], 16)
    assert s2[0, 0, 0] == 2.0 ** 120 and (c2[0, 0, :7] == c[0, 0, :7]).all()


def test_append_rounds_kept_values_below_the_normal_codes():
    """Scale 1, kept values of 2^-6 to 2^-9; a row of 896 doubles the scale, a
    small draft in its place brings a small one back, but not the bits."""
    kept = np.array([9, 15, 8, 16, 17, 1]) * 2.0 ** -9
    codes = serving.e4m3_encode(np.append(kept, [0.0, 0.0])).reshape(1, 1, 8, 1)
    assert codes.ravel()[:6].tolist() == [0x09, 0x0f, 0x08, 0x10, 0x10, 0x01]
    kept[4] = 16 * 2.0 ** -9  # 17 has five bits
    c, s = serving.append_q8(codes, np.ones((1, 1, 1)), [6], np.full((1, 1, 1, 1), 896.0), [1], 8)
    assert s[0, 0, 0] == 2.0
    lost = np.array([8, 16, 8, 16, 16, 0]) * 2.0 ** -9  # multiples of 2^-9 2, ties to even
    assert serving.values(c, s, 8).ravel()[:6].tolist() == lost.tolist()
    c, s = serving.append_q8(c, s, [6], np.full((1, 1, 1, 1), 0.5), [1], 8)
    assert s[0, 0, 0] == 2.0 ** -9
    assert serving.values(c, s, 8).ravel()[:6].tolist() == lost.tolist()


def test_append_keeps_values_of_normal_codes_exactly():
    """From 2^-6 of the new scale on every kept value survives any scale."""
    table = serving.e4m3_table()
    codes = np.arange(256, dtype=np.uint8)[np.isfinite(table)].reshape(1, 1, 254, 1)
    codes = np.concatenate([codes, np.zeros((1, 1, 2, 1), np.uint8)], 2)
    for k in range(12):
        c, s = serving.append_q8(codes, np.ones((1, 1, 1)), [254], np.full((1, 1, 1, 1), 448.0 * 2.0 ** k), [1], 256)
        assert s[0, 0, 0] == 2.0 ** k
        x, y = table[codes.ravel()[:254]], serving.values(c, s, 256).ravel()[:254]
        large = np.abs(x) >= 2.0 ** (k - 6)
        assert (x[large] == y[large]).all() and (np.abs(x - y) <= 2.0 ** (k - 10)).all()


# ----------------------------------------------------------------------------
# decode


def test_decode_refuses_more_rows_than_32_bits_count(lib):
    """2^32 query rows in units of a size that is allowed."""
    big = dict(q_blk=A, k_cache=2 * A, v_cache=3 * A, cache_len=6 * A, out=7 * A, lse=8 * A, B=512, Hq=64, Hkv=1,
               b=131000, d=32, intra_block_mode=0, stream=None, S_cap=1 << 18, workspace=9 * A, workspace_bytes=1 << 30)
    assert bd.bd_attn_decode_q8(**big, k_scale=4 * A, v_scale=5 * A, group=32) == bd.BD_ERR_UNSUPPORTED
    assert bd.bd_attn_decode(**big) == bd.BD_ERR_UNSUPPORTED
