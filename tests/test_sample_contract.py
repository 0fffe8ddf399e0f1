"""What include/peagle.h promises of the sampling calls' host side: what they refuse, before
anything is launched (no GPU)."""
import ctypes

import pytest

from test_oracle_kv_quant import A, pk  # noqa: F401 (A: an address that is never read, pk: fixture)

SAMPLE = dict(how=None, rows=3, vocab=100, logits=A, dtype=0, stride=0, u=A, d2t=A, token=A, prob=A,
              dist=A, errors=A)
VERIFY = dict(batch=2, K=3, tokens=A, how=None, vocab=100, target=A, dtype=1, stride=0, dv=50, draft=A,
              dist=A, d2t=A, u_accept=A, u_bonus=A, acc=A, bonus=A, prob=A, errors=A, work=A,
              bytes=8 * (32 + 512 * 12 + 16))


def _how(pk, **kw):  # noqa: F811
    return pk.PeagleSampling(**{**dict(temperature=A, top_k=A, top_p=A, min_p=A, rows_per=1), **kw})


def test_layouts(pk):  # noqa: F811
    assert ctypes.sizeof(pk.PeagleSampling) == 40 and pk.PeagleSampling.rows_per.offset == 32
    assert pk.DIST_BYTES == 32


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), "INVALID"), (dict(rows=-1), "INVALID"), (dict(vocab=0), "INVALID"),
    (dict(dtype=2), "INVALID"), (dict(dtype=-1), "INVALID"), (dict(logits=None), "INVALID"),
    (dict(logits=A + 2), "INVALID"), (dict(dtype=1, logits=A + 1), "INVALID"),
    (dict(stride=99), "INVALID"), (dict(stride=-100), "INVALID"), (dict(u=None), "INVALID"),
    (dict(u=A + 1), "INVALID"), (dict(token=None), "INVALID"), (dict(token=A + 2), "INVALID"),
    (dict(prob=A + 2), "INVALID"), (dict(dist=A + 4), "INVALID"), (dict(d2t=A + 1), "INVALID"),
    (dict(errors=A + 3), "INVALID"), (dict(vocab=262145), "UNSUPPORTED"),
    (dict(rows=(1 << 24) + 1), "UNSUPPORTED")])
def test_sample_refuses(pk, kw, code):  # noqa: F811
    args = {**SAMPLE, **kw}
    assert pk.lib().peagle_sample(*args.values(), None) == getattr(pk, "PEAGLE_ERR_" + code)


@pytest.mark.parametrize("kw", [dict(rows_per=-1), dict(temperature=A + 1), dict(top_k=A + 2),
                                dict(top_p=A + 3), dict(min_p=A + 2)])
def test_settings_are_refused(pk, kw):  # noqa: F811
    how, bad = _how(pk, **kw), pk.PEAGLE_ERR_INVALID
    assert pk.lib().peagle_sample(*{**SAMPLE, "how": how}.values(), None) == bad
    assert pk.lib().peagle_verify_sample(*{**VERIFY, "how": how}.values(), None) == bad


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), "INVALID"), (dict(K=0), "INVALID"), (dict(K=65), "CAPACITY"),
    (dict(vocab=0), "INVALID"), (dict(vocab=262145), "UNSUPPORTED"), (dict(dv=0), "INVALID"),
    (dict(dv=262145), "UNSUPPORTED"), (dict(dtype=3), "INVALID"), (dict(stride=99), "INVALID"),
    (dict(draft=None), "INVALID"), (dict(dist=None), "INVALID"), (dict(draft=A + 2), "INVALID"),
    (dict(dist=A + 4), "INVALID"), (dict(work=A + 8), "INVALID"), (dict(bytes=8 * (32 + 512 * 12 + 16) - 1), "CAPACITY"),
    (dict(batch=1 << 23), "UNSUPPORTED"), (dict(target=None), "INVALID"), (dict(target=A + 1), "INVALID"),
    *[({k: None}, "INVALID") for k in ("tokens", "u_accept", "u_bonus", "acc", "bonus", "work")],
    *[({k: A + 2}, "INVALID") for k in ("tokens", "u_accept", "u_bonus", "acc", "bonus", "prob", "errors",
                                        "d2t")]])
def test_verify_refuses(pk, kw, code):  # noqa: F811
    args = {**VERIFY, **kw}
    assert pk.lib().peagle_verify_sample(*args.values(), None) == getattr(pk, "PEAGLE_ERR_" + code)


def test_workspace_sizes(pk):  # noqa: F811
    f = pk.lib().peagle_verify_sample_workspace
    row = 32 + 512 * 12 + 16  # a record, and a list of up to 512 tokens
    assert f(2, 3, 100) == 8 * row and f(1, 64, 262144) == 65 * row
    assert f(8192, 1, 100) == 16384 * row and f(8193, 1, 100) == 16386 * 32  # no lists
    assert f(0, 3, 100) == f(1, 0, 100) == f(1, 1, 0) == pk.PEAGLE_ERR_INVALID
    assert f(1, 65, 100) == pk.PEAGLE_ERR_CAPACITY and f(1, 1, 262145) == pk.PEAGLE_ERR_UNSUPPORTED
    with pytest.raises(pk.PeagleError, match="32 bits"):
        pk.peagle_verify_sample_workspace(1 << 32, 1, 100)
    with pytest.raises(pk.PeagleError):
        pk.peagle_verify_sample_workspace(0, 1, 100)


def test_the_binding_refuses_what_is_not_on_the_gpu(pk):  # noqa: F811
    torch = pytest.importorskip("torch")
    f = torch.zeros(3, 8)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(pk.PeagleError, match="not the current CUDA device"):
        pk.peagle_sample(None, f, f[:, 0].contiguous(), i)
    for bad in (f.half(), f.long(), f[0], f[:, ::2], f[:1].expand(3, 8)):
        with pytest.raises(pk.PeagleError):
            pk.peagle_sample(None, bad, f[:, 0].contiguous(), i)
    for kw in (dict(temperature=f[:, ::2]), dict(temperature=i), dict(top_k=f),
               dict(temperature=f[:, 0].contiguous(), top_k=i[:2]), dict(rows_per=0)):
        with pytest.raises(pk.PeagleError):
            pk.sampling_struct(**kw)
