"""Pins of the 8-bit cache's oracle (no GPU), and the refusals of its calls before anything is
launched: e4m3 rounding against torch's conversion, the scale's definition, append in one piece
and in several, attention against the draft pass's attention and by joining two halves."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv_quant_oracle as Q
from oracle import peagle_oracle as O


def test_e4m3_round_is_torchs_conversion():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    fine = codes[np.isfinite(codes)]
    assert len(fine) == 254 and fine.max() == Q.TOP
    assert np.array_equal(Q.e4m3_round(fine), fine)
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.float16).double()
    x = x[x.abs() <= Q.TOP]  # every f16 value in range: ties and subnormals among them
    assert len(x) > 40000
    want = x.float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(Q.e4m3_round(x.numpy()), want)


def test_scale_is_the_smallest_power_of_two():
    r = np.random.default_rng(1)
    a = np.concatenate([2.0 ** r.uniform(-30, 120, 500), 448.0 * 2.0 ** np.arange(-20, 100.0),
                        np.nextafter(448.0 * 2.0 ** np.arange(-20, 100.0), np.inf)])
    s = Q.block_scale(a)
    assert (a <= Q.TOP * s).all() and (a > Q.TOP * s / 2).all()
    assert (np.frexp(s)[0] == 0.5).all()
    assert Q.block_scale(0.0) == 1.0 and Q.block_scale(1e-30) == 2.0 ** Q.E_MIN


@pytest.mark.parametrize("block", [16, 32])
def test_append_in_pieces_equals_append_at_once(block):
    """Rows of a narrow range (nothing falls below the smallest codes when a scale grows) give the
    same cache however they are cut, and rows dropped in between leave no trace."""
    r = np.random.default_rng(2)
    L, B, H, hd, cap = 2, 2, 3, 64, 96
    rows = r.uniform(0.5, 4.0, (L, B, 70, H, hd)) * r.choice([-1.0, 1.0], (L, B, 70, H, hd))
    codes, scale = np.zeros((L, B, H, cap, hd)), np.ones((L, B, H, cap // block))
    whole = Q.append(codes, scale, block, [0, 0], [70, 70], rows)
    c, s, at = codes, scale, 0
    for n in (1, 5, 26, 7, 31):
        c, s = Q.append(c, s, block, [at] * 2, [n + 3] * 2, 50.0 * rows[:, :, :n + 3])
        c, s = Q.append(c, s, block, [at] * 2, [n] * 2, rows[:, :, at:at + n])
        at += n
    assert at == 70
    blocks = -(-70 // block)
    assert np.array_equal(s[..., :blocks], whole[1][..., :blocks])
    assert np.array_equal(c[..., :70, :], whole[0][..., :70, :])
    err = np.abs(Q.values(*whole, block)[..., :70, :] - np.swapaxes(rows, 2, 3))
    assert (err <= 2.0 ** -4 * np.abs(np.swapaxes(rows, 2, 3))).all()


def test_attention_is_the_draft_pass_attention_and_joins():
    r = np.random.default_rng(3)
    B, K, nq, H, hd, cap = 2, 3, 4, 2, 64, 40
    q = r.standard_normal((B * K, nq, hd))
    k, v = r.standard_normal((2, B, H, cap, hd))
    lens = [0, 30]
    out, lse, _ = Q.attention(q, k, v, lens, K)
    for b in range(B):
        for j in range(K):
            for h in range(nq):
                n = lens[b] + j + 1
                want = O.attend(q[b * K + j, h], k[b, h // 2, :n], v[b, h // 2, :n], hd ** -0.5)
                assert np.allclose(out[b * K + j, h], want, rtol=0, atol=1e-12)
    # the slots before 12 and the 18 after them, joined by lse, are the 30 of request 1
    whole, wl, _ = Q.attention(q, k, v, [30, 30], K, causal=False)
    a, la, _ = Q.attention(q, k, v, [12, 12], K, causal=False)
    c, lc, _ = Q.attention(q, k[:, :, 12:], v[:, :, 12:], [18, 18], K, causal=False)
    both = np.logaddexp(la, lc)
    assert np.allclose(both, wl, rtol=0, atol=1e-12)
    got = a * np.exp(la - both)[..., None] + c * np.exp(lc - both)[..., None]
    assert np.allclose(got, whole, rtol=0, atol=1e-12)
    none, ln, _ = Q.attention(q, k, v, [0, 0], K, causal=False)
    assert not none.any() and (ln == -np.inf).all()
    # a window of one position sees the row's own slot
    one, _, _ = Q.attention(q, k, v, lens, K, window=1)
    assert np.array_equal(one[K, 0], v[1, 0, 30])


# ---- refusals on the host (no GPU: pointers are never followed) -------------------------

@pytest.fixture(scope="module")
def pk():
    from drafting_eagle_draft_gb300 import build

    build.build()
    import drafting_eagle_draft_gb300 as pk

    pk.lib()
    return pk


A = 1 << 20  # an aligned address that nothing follows


def _kv(pk, **kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, errors=None, n_layers=2, batch=3, n_kv_heads=2,
             capacity=64, head_dim=64, block=32)
    d.update(kw)
    return pk.PeagleKVQuant(**d)


def _rows(pk, **kw):
    d = dict(k=A, v=A, layer_stride=4096, batch_stride=1024, token_stride=128, head_stride=64,
             dtype=pk.PEAGLE_BF16)
    d.update(kw)
    return pk.PeagleKVRows(**d)


def test_struct_layouts(pk):
    assert ctypes.sizeof(pk.PeagleKVQuant) == 5 * 8 + 6 * 4
    assert ctypes.sizeof(pk.PeagleKVRows) == 7 * 8
    assert pk.PeagleKVQuant.block.offset == 60 and pk.PeagleKVRows.dtype.offset == 48


CACHE = [
    (dict(k=None), "INVALID"), (dict(v_scale=None), "INVALID"), (dict(k=A + 8), "INVALID"),
    (dict(v=A + 1), "INVALID"), (dict(k_scale=A + 2), "INVALID"), (dict(errors=A + 2), "INVALID"),
    (dict(capacity=65), "INVALID"), (dict(capacity=0), "INVALID"), (dict(n_layers=0), "INVALID"),
    (dict(n_layers=65536), "INVALID"), (dict(n_kv_heads=0), "INVALID"), (dict(batch=2), "CAPACITY"),
    (dict(capacity=-32), "INVALID"), (dict(head_dim=96), "UNSUPPORTED"),
    (dict(block=8), "UNSUPPORTED"), (dict(block=48), "UNSUPPORTED"), (dict(block=0), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,code", CACHE)
def test_every_call_refuses_a_bad_cache(pk, kw, code):
    L, kv, rows = pk.lib(), _kv(pk, **kw), _rows(pk)
    code = getattr(pk, "PEAGLE_ERR_" + code)
    assert L.peagle_append_kv_quant(kv, -1, 3, A, A + 64, 0, rows, 4, 1, None) == code
    assert L.peagle_read_kv_quant(kv, -1, 3, None, A, rows, 4, None) == code
    assert L.peagle_decode_attention_quant_workspace(kv, 3, 2, 4) == code
    assert L.peagle_decode_attention_quant(kv, 0, 3, 2, 4, A, pk.PEAGLE_BF16, 0, A, 1, 0, 0.125, A,
                                           None, A, 1 << 40, None) == code


def test_append_and_read_refuse(pk):
    L, kv, rows = pk.lib(), _kv(pk), _rows(pk)
    bad, cap, uns = pk.PEAGLE_ERR_INVALID, pk.PEAGLE_ERR_CAPACITY, pk.PEAGLE_ERR_UNSUPPORTED

    def append(layer=-1, batch=3, lens=A, n=A + 64, extra=0, rows=rows, n_max=4, adv=1):
        return L.peagle_append_kv_quant(kv, layer, batch, lens, n, extra, rows, n_max, adv, None)

    def read(layer=-1, batch=3, counts=A, rows=rows, n_max=4):
        return L.peagle_read_kv_quant(kv, layer, batch, None, counts, rows, n_max, None)

    for f in (append, read):
        assert f(layer=-2) == bad and f(layer=2) == bad
        assert f(batch=0) == bad and f(batch=4) == cap
        assert f(n_max=0) == bad and f(n_max=(1 << 30) + 1) == bad
        for kw in (dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 2), dict(token_stride=100),
                   dict(layer_stride=4), dict(batch_stride=-12), dict(head_stride=1)):
            assert f(rows=_rows(pk, **kw)) == bad, kw
        assert f(rows=_rows(pk, dtype=7)) == uns
        assert f(rows=None) == bad
        # 16 bytes are 4 elements in fp32
        assert f(rows=_rows(pk, dtype=pk.PEAGLE_F32, token_stride=66)) == bad
    assert append(lens=None) == bad and append(adv=2) == bad
    assert append(n=A) == bad  # n_commit is the buffer that advances
    assert append(extra=5) == bad and append(extra=-5) == bad
    assert read(counts=None) == bad


def test_attention_refuses(pk):
    L, kv = pk.lib(), _kv(pk)
    bad, cap, uns = pk.PEAGLE_ERR_INVALID, pk.PEAGLE_ERR_CAPACITY, pk.PEAGLE_ERR_UNSUPPORTED

    def call(layer=0, batch=3, K=2, nq=4, q=A, dtype=pk.PEAGLE_BF16, stride=0, lens=A, causal=1,
             window=0, scale=0.125, out=A, lse=None, work=A, n=1 << 40):
        return L.peagle_decode_attention_quant(kv, layer, batch, K, nq, q, dtype, stride, lens,
                                               causal, window, scale, out, lse, work, n, None)

    for kw in (dict(layer=-1), dict(layer=2), dict(batch=0), dict(K=0), dict(nq=0), dict(nq=3),
               dict(q=None), dict(q=A + 8), dict(stride=12), dict(lens=None), dict(causal=2),
               dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(out=None),
               dict(out=A + 4), dict(lse=A + 2), dict(work=None), dict(work=A + 64)):
        assert call(**kw) == bad, kw
    assert call(dtype=7) == uns
    assert call(K=16, nq=18) == uns and call(K=129, nq=2) == uns
    assert call(batch=4) == cap
    # (slots of a layer beyond what the walk over them counts)
    big = _kv(pk, batch=65535, n_kv_heads=16, capacity=1 << 15)
    assert L.peagle_decode_attention_quant(big, 0, 65535, 2, 16, A, pk.PEAGLE_BF16, 0, A, 1, 0,
                                           0.125, A, None, A, 1 << 40, None) == uns
    need = L.peagle_decode_attention_quant_workspace(kv, 3, 2, 4)
    assert need > 0 and call(n=need - 1) == cap and call(n=0) == cap


def test_binding_refuses_tensors_that_do_not_fit(pk):
    k = torch.zeros(1, 2, 2, 64, 64, dtype=torch.uint8)
    s = torch.zeros(1, 2, 2, 2)
    kv = pk.kv_quant_struct(k, k.clone(), s, s.clone())
    assert kv.block == 32 and kv.capacity == 64
    for args in ((k, k, s[..., :1], s), (k.float(), k, s, s), (k, k[:, :1], s, s),
                 (k.transpose(1, 2), k, s, s), (k[0], k, s, s), (k, k, s.double(), s),
                 (k, k, s[..., :0], s)):
        with pytest.raises(pk.PeagleError):
            pk.kv_quant_struct(*args)
    with pytest.raises(pk.PeagleError):
        pk.kv_quant_struct(k, k, s, s, torch.zeros(1))
    # a cache on the CPU never reaches a kernel
    rows = torch.zeros(1, 2, 4, 2, 64)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(pk.PeagleError):
        pk.peagle_append_kv_quant(kv, 2, n, n.clone(), rows, rows, 4, stream=0)
    with pytest.raises(pk.PeagleError):
        pk.peagle_read_kv_quant(kv, 2, n, rows, rows, 4, stream=0)
    q = torch.zeros(4, 2, 64)
    with pytest.raises(pk.PeagleError):
        pk.peagle_decode_attention_quant(kv, 0, 2, 2, 2, q, n, q, torch.zeros(256), stream=0)
