"""What include/peagle.h promises of the shared-prefix attention's host side, before anything is
launched (no GPU), and pins of its fp64 oracle."""
import numpy as np
import pytest

from oracle import kv_quant_oracle as Q
from oracle import shared_attn_oracle as S
from test_oracle_kv_quant import A, pk  # noqa: F401 (A: an address that is never read, pk: fixture)

CALL = dict(dtype=1, batch=2, K=3, nq=8, nkv=2, hd=64, q=A, stride=0, pk=A, pv=A, pcap=100, plen=A, k=A, v=A, cap=50,
            lens=A, causal=1, scale=0.125, out=A << 4, lse=A, errors=A, work=A, bytes=1 << 40)
SIZES = ("dtype", "batch", "K", "nq", "nkv", "hd", "pcap", "cap")
BAD_SIZES = [
    (dict(dtype=2), "INVALID"), (dict(batch=0), "INVALID"), (dict(K=0), "INVALID"), (dict(nq=0), "INVALID"),
    (dict(nkv=0), "INVALID"), (dict(nq=7), "INVALID"), (dict(pcap=0), "INVALID"), (dict(cap=0), "INVALID"),
    (dict(hd=96), "UNSUPPORTED"), (dict(hd=0), "UNSUPPORTED"), (dict(K=33), "UNSUPPORTED"),
    (dict(batch=1 << 22), "UNSUPPORTED"), (dict(pcap=(1 << 24) + 1), "UNSUPPORTED"),
    (dict(cap=(1 << 24) + 1), "UNSUPPORTED"), (dict(nkv=65536, nq=65536, K=1, batch=1), "UNSUPPORTED")]


@pytest.mark.parametrize("kw,code", BAD_SIZES + [
    *[({k: None}, "INVALID") for k in ("q", "pk", "pv", "plen", "k", "v", "lens", "out", "work")],
    *[({k: A + 8}, "INVALID") for k in ("q", "pk", "pv", "k", "v", "work")],
    *[({k: A + 2}, "INVALID") for k in ("plen", "lens", "lse", "errors")],
    (dict(out=(A << 4) + 8), "INVALID"), (dict(work=A + 128), "INVALID"), (dict(stride=511), "INVALID"),
    (dict(stride=513), "INVALID"), (dict(causal=2), "INVALID"), (dict(scale=float("nan")), "INVALID"),
    (dict(scale=float("inf")), "INVALID"), (dict(scale=3e38), "INVALID"), (dict(out=A), "INVALID"),
    (dict(out=A + 5 * 1024), "INVALID"), (dict(bytes=0), "CAPACITY")])
def test_the_call_refuses(pk, kw, code):  # noqa: F811
    f, code = pk.lib().peagle_decode_attention_shared, getattr(pk, "PEAGLE_ERR_" + code)
    for dtype in (0, 1):
        if "dtype" in kw and dtype:
            continue
        args = {**CALL, "dtype": dtype, **kw}
        if dtype == 0 and kw in (dict(stride=513), dict(stride=511)):
            args["stride"] = 514 if kw["stride"] == 513 else 511
        assert f(*args.values(), None) == code


@pytest.mark.parametrize("kw,code", BAD_SIZES)
def test_the_workspace_refuses(pk, kw, code):  # noqa: F811
    args = {k: {**CALL, **kw}[k] for k in SIZES}
    assert pk.lib().peagle_decode_attention_shared_workspace(*args.values()) == getattr(pk, "PEAGLE_ERR_" + code)


def test_workspace_is_exactly_what_is_wanted(pk):  # noqa: F811
    L = pk.lib()
    for dtype in (0, 1):
        need = L.peagle_decode_attention_shared_workspace(*[{**CALL, "dtype": dtype}[k] for k in SIZES])
        assert need > 0
        args = {**CALL, "dtype": dtype, "bytes": need - 1}
        assert L.peagle_decode_attention_shared(*args.values(), None) == pk.PEAGLE_ERR_CAPACITY


def test_the_wait_drill_refuses_other_waits(pk):  # noqa: F811
    for wait in (-2, 6):
        assert pk.lib().peagle_set_wait_limit_shared(0, wait) == pk.PEAGLE_ERR_INVALID
    with pytest.raises(pk.PeagleError):
        pk.peagle_set_wait_limit_shared(0, 1 << 33)
    pk.peagle_set_wait_limit_shared(0, -1)


def test_the_binding_refuses_tensors_that_do_not_fit(pk):  # noqa: F811
    import torch

    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype)

    q, p, k, n = t(6, 8, 64), t(2, 100, 64), t(2, 2, 50, 64), t(2, dtype=torch.int32)
    need = pk.peagle_decode_attention_shared_workspace(2, 3, q, p, k)
    w = torch.zeros(need, dtype=torch.uint8)
    for bad in ((q.half(), p, k), (t(5, 8, 64), p, k), (q, t(3, 100, 64), k), (q, p, t(1, 2, 50, 64)),
                (q, t(2, 100, 128), k), (q[0], p, k)):
        with pytest.raises(pk.PeagleError):
            pk.peagle_decode_attention_shared_workspace(2, 3, *bad)
    with pytest.raises(pk.PeagleError, match="not the current CUDA device"):
        pk.peagle_decode_attention_shared(2, 3, q, p, p, n, k, k, n, q.clone(), w)


def test_oracle_is_attention_over_both_and_joins():
    """Against the 8-bit cache's oracle on the whole rows, and joined from the prefix's and the
    requests' own parts by the log-sum-exp."""
    r = np.random.default_rng(1)
    B, K, nq, nkv, hd, P, cap = 2, 3, 4, 2, 64, 9, 20
    lens = [4, 0]
    q, p, pv = r.standard_normal((B * K, nq, hd)), *r.standard_normal((2, nkv, 12, hd))
    k, v = r.standard_normal((2, B, nkv, cap, hd))
    for causal in (True, False):
        out, lse, _ = S.attention(q, p, pv, P, k, v, lens, K, causal)
        both = [np.concatenate([np.repeat(x[None, :, :P], B, 0), y], 2) for x, y in ((p, k), (pv, v))]
        want, wl, _ = Q.attention(q, *both, [P + n for n in lens], K, causal=causal)
        assert np.allclose(out, want, rtol=0, atol=1e-12) and np.allclose(lse, wl, rtol=0, atol=1e-12)
        a, la, _ = S.attention(q, p, pv, P, k, v, [0, 0], K, False)
        c, lc, _ = S.attention(q, p, pv, 0, k, v, lens, K, causal)
        got = a * np.exp(la - lse)[..., None] + c * np.exp(lc - lse)[..., None]
        assert np.allclose(got, out, rtol=0, atol=1e-12)
    none, ln, _ = S.attention(q, p, pv, 0, k, v, [0, 0], K, False)
    assert not none.any() and (ln == -np.inf).all()


def test_work_beyond_31_bits_is_refused(pk):  # noqa: F811
    """What a bf16 call divides among CTAs is counted in 32 bits; a call that is larger is refused, by the
    workspace's size too, and one that is not is taken."""
    size, call = pk.lib().peagle_decode_attention_shared_workspace, pk.lib().peagle_decode_attention_shared
    most = dict(dtype=1, batch=4096, K=8, nq=64, nkv=64, hd=64, pcap=1 << 24, cap=1 << 20)
    assert size(*most.values()) == pk.PEAGLE_ERR_UNSUPPORTED
    assert call(*{**CALL, **most, "out": 1 << 60}.values(), None) == pk.PEAGLE_ERR_UNSUPPORTED
    assert size(*{**most, "batch": 64}.values()) > 0 and size(*{**most, "dtype": 0}.values()) > 0
