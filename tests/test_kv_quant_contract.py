"""What include/peagle.h promises of the 8-bit cache's host side, and of its values by the fp64
oracle (no GPU)."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import kv_quant_oracle as Q
from test_oracle_kv_quant import A, CACHE, _kv, _rows, pk  # noqa: F401 (pk: fixture)


def test_a_dropped_draft_rounds_committed_slots_unless_they_are_restored():
    """Why peagle_save_kv_quant is there: 8 committed rows, one draft row with an element of 3e4,
    dropped, and a quiet row; against the cache that never saw the draft."""
    r = np.random.default_rng(4)
    block, hd = 32, 64
    rows = r.standard_normal((1, 1, 8, 1, hd))
    loud, quiet = r.standard_normal((2, 1, 1, 1, 1, hd))
    loud[..., 5] = 3e4
    empty = np.zeros((1, 1, 1, 64, hd)), np.ones((1, 1, 1, 2))
    one = Q.append(*empty, block, [0], [8], rows)
    never = Q.append(*one, block, [8], [1], quiet)
    drafted = Q.append(*one, block, [8], [1], loud)
    traced = Q.append(*drafted, block, [8], [1], quiet)
    assert np.array_equal(traced[1], never[1])  # the scale comes back, the values do not
    assert (traced[0] != never[0])[..., :8, :].mean() > 0.5
    codes, scale = drafted[0].copy(), drafted[1].copy()  # restored: the open block's committed part
    codes[..., :8, :], scale[..., 0] = one[0][..., :8, :], one[1][..., 0]
    clean = Q.append(codes, scale, block, [8], [1], quiet)
    assert np.array_equal(clean[0][..., :9, :], never[0][..., :9, :])
    assert np.array_equal(clean[1], never[1])


@pytest.mark.parametrize("kw,code", CACHE)
def test_save_and_restore_refuse_a_bad_cache(pk, kw, code):  # noqa: F811
    L, kv, code = pk.lib(), _kv(pk, **kw), getattr(pk, "PEAGLE_ERR_" + code)
    for f in (L.peagle_save_kv_quant, L.peagle_restore_kv_quant):
        assert f(kv, -1, 3, A, A, 1 << 50, None) == code
    if kw != dict(batch=2):
        assert L.peagle_save_kv_quant_bytes(kv) == code


def test_save_and_restore_refuse(pk):  # noqa: F811
    L, kv = pk.lib(), _kv(pk)
    bad, cap = pk.PEAGLE_ERR_INVALID, pk.PEAGLE_ERR_CAPACITY
    need = pk.peagle_save_kv_quant_bytes(kv)
    assert need == 2 * 2 * 3 * 2 * (32 * 64 + 4)
    for f in (L.peagle_save_kv_quant, L.peagle_restore_kv_quant):
        for layer in (-2, 2):
            assert f(kv, layer, 3, A, A, need, None) == bad
        assert f(kv, -1, 0, A, A, need, None) == bad and f(kv, -1, 4, A, A, need, None) == cap
        assert f(kv, -1, 3, None, A, need, None) == bad
        assert f(kv, -1, 3, A, None, need, None) == bad
        assert f(kv, -1, 3, A, A + 8, need, None) == bad
        assert f(kv, -1, 3, A, A, need - 1, None) == cap and f(kv, 1, 3, A, A, 0, None) == cap
    huge = _kv(pk, n_layers=65535, batch=65535, n_kv_heads=65535)
    assert L.peagle_save_kv_quant_bytes(huge) == pk.PEAGLE_ERR_UNSUPPORTED


def test_repeated_growth_keeps_the_documented_bound():
    """A value is encoded again whenever its block's scale grows: 29.125 x 2^-9 beside 448 is 30 x
    2^-9, beside 897 it is 32 x 2^-9, off by 1.4 times what one encoding would allow."""
    block, hd = 16, 64
    c = np.zeros((1, 1, 1, 16, hd)), np.ones((1, 1, 1, 1))
    x = 29.125 * 2.0 ** -9
    for at, top in enumerate((448.0, 449.0, 897.0)):
        row = np.zeros((1, 1, 1, 1, hd))
        row[..., 0], row[..., 1] = top, x
        c = Q.append(*c, block, [at], [1], row)
    err, s = abs(Q.values(*c, block)[0, 0, 0, 0, 1] - x), c[1].max()
    assert max(2.0 ** -4 * x, 2.0 ** -10 * s) < err <= 2.0 ** -4 * x + 2.0 ** -9 * s
    assert s * 2.0 ** -9 <= 2.0 ** -16.8 * 897.0


@pytest.mark.parametrize("grow", [0.3, 1.0, 2.7])
def test_rows_appended_one_by_one_against_the_rows_themselves(grow):
    r = np.random.default_rng(int(10 * grow))
    block, hd, n = 32, 64, 32
    rows = r.standard_normal((1, 1, n, 2, hd)) * 2.0 ** (grow * np.arange(n))[:, None, None]
    c = np.zeros((1, 1, 2, 32, hd)), np.ones((1, 1, 2, 1))
    for at in range(n):
        c = Q.append(*c, block, [at], [1], rows[:, :, at:at + 1])
        x = np.swapaxes(rows[:, :, :at + 1], 2, 3)
        err = np.abs(Q.values(*c, block)[..., :at + 1, :] - x)
        assert (err <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * c[1][..., None]).all()


def test_a_block_below_the_smallest_scale_keeps_half_of_its_spacing():
    x = np.full((1, 1, 1, 1, 64), 2.0 ** -48)
    codes, scale = Q.append(np.zeros((1, 1, 1, 16, 64)), np.ones((1, 1, 1, 1)), 16, [0], [1], x)
    assert scale[0, 0, 0, 0] == 2.0 ** -40
    assert (np.abs(codes[..., 0, :] * scale - 2.0 ** -48) <= 2.0 ** -50).all()


def test_wait_limit_refuses_an_unknown_wait(pk):  # noqa: F811
    for w in (-2, 9, 1000):
        with pytest.raises(pk.PeagleError) as e:
            pk.peagle_set_wait_limit_quant(1000, w)
        assert e.value.code == pk.PEAGLE_ERR_INVALID
    pk.peagle_set_wait_limit_quant(0, -1)


def test_host_calls_work_without_torch(pk):  # noqa: F811
    """The package imports, and its host-only calls answer, where torch cannot be imported."""
    root = os.path.dirname(os.path.dirname(pk.LIB_PATH))
    code = ("import sys; sys.modules['torch'] = None\n"
            "import drafting_eagle_draft_gb300 as m\n"
            "assert m.strerror(m.PEAGLE_ERR_CAPACITY) and m.lib().peagle_status(None) == m.PEAGLE_ERR_INVALID\n"
            "kv = m.PeagleKVQuant(k=1 << 20, v=1 << 20, k_scale=1 << 20, v_scale=1 << 20, n_layers=1,\n"
            "                     batch=1, n_kv_heads=1, capacity=64, head_dim=64, block=32)\n"
            "assert m.peagle_decode_attention_quant_workspace(kv, 1, 1, 1) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_a_cache_filled_by_hand_is_refused_by_the_tensor_calls(pk):  # noqa: F811
    kv = _kv(pk)
    for call in (lambda: pk.peagle_append_kv_quant(kv, 1, None, None, None, None, 1, stream=0),
                 lambda: pk.peagle_read_kv_quant(kv, 1, None, None, None, 1, stream=0),
                 lambda: pk.peagle_save_kv_quant(kv, 1, None, None, stream=0),
                 lambda: pk.peagle_restore_kv_quant(kv, 1, None, None, stream=0),
                 lambda: pk.peagle_decode_attention_quant(kv, 0, 1, 1, 1, None, None, None, None,
                                                          stream=0)):
        with pytest.raises(pk.PeagleError) as e:
            call()
        assert e.value.code == pk.PEAGLE_ERR_INVALID


def test_whole_numbers_beyond_32_bits_are_refused(pk):  # noqa: F811
    """ctypes passes their low 32 bits: 2^32 + 1 draft rows came in as one."""
    kv = _kv(pk)
    assert pk.peagle_decode_attention_quant_workspace(kv, 3, 2, 4) > 0
    for args in ((3 + 2 ** 32, 2, 4), (3, 1 + 2 ** 32, 4), (3, 2, 4 - 2 ** 32)):
        with pytest.raises(pk.PeagleError):
            pk.peagle_decode_attention_quant_workspace(kv, *args)
    with pytest.raises(pk.PeagleError):
        pk.peagle_set_wait_limit_quant(0, 2 ** 32 - 1)


def test_attention_refuses_a_scale_that_log2_e_makes_infinite(pk):  # noqa: F811
    L, kv = pk.lib(), _kv(pk)
    for scale in (2.5e38, -3e38):
        assert L.peagle_decode_attention_quant(kv, 0, 3, 2, 4, A, pk.PEAGLE_BF16, 0, A, 1, 0, scale, A,
                                               None, A, 1 << 40, None) == pk.PEAGLE_ERR_INVALID


def test_attention_refuses_an_output_over_its_queries(pk):  # noqa: F811
    L, kv, row = pk.lib(), _kv(pk), 4 * 64 * 2  # six rows of four heads of 64, bf16
    bad = pk.PEAGLE_ERR_INVALID

    def call(out, stride=0):
        return L.peagle_decode_attention_quant(kv, 0, 3, 2, 4, A, pk.PEAGLE_BF16, stride, A, 1, 0, 0.125,
                                               out, None, A, 1 << 40, None)

    for out in (A, A + 16, A + 6 * row - 16, A - 6 * row + 16):
        assert call(out) == bad
    # three halves of a row apart, and half a row backwards
    assert call(A + 8 * row, 3 * 4 * 64 // 2) == bad and call(A - 5 * row, -4 * 64 // 2) == bad


def test_read_refuses_keys_and_values_into_the_same_rows(pk):  # noqa: F811
    assert pk.lib().peagle_read_kv_quant(_kv(pk), -1, 3, None, A, _rows(pk), 4,
                                         None) == pk.PEAGLE_ERR_INVALID
