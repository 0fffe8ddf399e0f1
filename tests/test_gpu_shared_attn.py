"""Decode attention over a shared prefix on the GPU against its fp64 oracle.

Bounds.  fp32: scores are sums of head_dim products of unit size and their maximum, exponentials and
sums of n terms follow, each rounded by 2^-24: with scores up to 8 here, a weight is off by at most
(head_dim + 16) 2^-24 x 8 of itself, and so is the sum; the output by twice that of its size (the sum
of |weight x value|).  bf16 has 7 fraction bits: the spacing at 1 is 2^-7 and a rounding is off by at
most 2^-8 of the value.  The weights are rounded so, and then the result, which may be (1 + 2^-8) of
its size: 2^-8 + 2^-8 (1 + 2^-8) together, and the fp32 part as above."""
import numpy as np
import pytest
import torch

from oracle import shared_attn_oracle as A
from pe_helpers import pk

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def ints(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


class Call:
    def __init__(self, dtype, B, K, nq, nkv, hd, prefix, lens, causal=True, seed=1, pcap=None, cap=None, scale=None,
                 spare=float("nan")):
        r = np.random.default_rng(seed)
        self.B, self.K, self.causal, self.scale, self.prefix, self.lens = B, K, causal, scale, prefix, list(lens)
        pcap = pcap or prefix + 3
        cap = cap or max(list(lens) + [0]) + (K if causal else 0) + 2
        t = DT[dtype]

        def rows(*shape):
            return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).cuda().to(t)

        self.q, self.pk, self.pv = rows(B * K, nq, hd), rows(nkv, pcap, hd), rows(nkv, pcap, hd)
        self.k, self.v = rows(B, nkv, cap, hd), rows(B, nkv, cap, hd)
        # slots that no row sees
        self.pk[:, prefix:], self.pv[:, prefix:] = spare, spare
        for b, n in enumerate(lens):
            end = max(0, n) + (K if causal else 0)
            self.k[b, :, end:], self.v[b, :, end:] = spare, spare
        self.errors = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full((B * K, nq, hd), 7.0, device="cuda", dtype=t)
        self.lse = torch.full((B * K, nq), 7.0, device="cuda")
        self.plen, self.slens = ints([prefix]), ints(lens)
        self.work = torch.full((pk().peagle_decode_attention_shared_workspace(B, K, self.q, self.pk, self.k),), 0xff,
                               dtype=torch.uint8, device="cuda")

    def run(self, **kw):
        a = dict(out_lse=self.lse, causal=self.causal, scale=self.scale, errors=self.errors)
        a.update(kw)
        pk().peagle_decode_attention_shared(self.B, self.K, self.q, self.pk, self.pv, self.plen, self.k, self.v,
                                            self.slens, self.out, self.work, **a)
        return self.out.clone(), self.lse.clone()

    def host(self):
        return [x.float().cpu().double().numpy() for x in (self.q, self.pk, self.pv, self.k, self.v)]

    def want(self):
        q, p, pv, k, v = self.host()
        return A.attention(q, p, pv, self.prefix, k, v, self.lens, self.K, self.causal, self.scale)


def bounds(c, lse, size):
    hd = c.q.shape[-1]
    top = max(8.0, float(np.abs(lse[np.isfinite(lse)]).max(initial=0)))
    f32 = 2 * (hd + 16) * 2.0 ** -24 * top
    return ((2.0 ** -7 + 2.0 ** -16 if c.q.dtype is torch.bfloat16 else 0) + f32) * size + 2.0 ** -24 * size, f32


def check(c):
    got, glse = c.run()
    assert c.errors.item() == 0
    out, lse, size = c.want()
    tol, ltol = bounds(c, lse, size)
    g = got.float().cpu().double().numpy()
    assert np.array_equal(np.isinf(glse.cpu().numpy()), np.isinf(lse))
    seen = np.isfinite(lse)
    assert np.abs(glse.cpu().double().numpy()[seen] - lse[seen]).max(initial=0) <= ltol
    assert not g[~seen].any()
    assert (np.abs(g - out) <= tol).all(), np.max(np.abs(g - out) / np.maximum(tol, 1e-300))
    again, _ = c.run()
    assert torch.equal(again, got)


SHAPES = [  # B, K, nq, nkv, prefix, lens
    (1, 1, 1, 1, 1, [0]),
    (1, 1, 1, 1, 0, [0]),
    (2, 4, 4, 2, 128, [5, 16]),
    (1, 8, 64, 8, 129, [127]),
    (3, 5, 6, 2, 77, [1, 0, 30]),
    (5, 3, 14, 2, 640, [0, 125, 126, 127, 300]),
    (4, 8, 32, 4, 257, [13, 255, 256, 60]),     # two row tiles a head
    (9, 16, 16, 2, 300, [7 * i for i in range(9)]),  # nine: an odd one
    (40, 1, 8, 4, 1000, list(range(40))),
    (33, 2, 2, 1, 5, [0] * 33),
    (2, 7, 16, 1, 3000, [700, 33]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention(shape, causal, hd, dtype):
    B, K, nq, nkv, prefix, lens = shape
    check(Call(dtype, B, K, nq, nkv, hd, prefix, lens, causal))


def check_rows(c, rows=None):
    """As check, of some rows; the values that a row sees may be NaN or infinite in places."""
    got, _ = c.run()
    assert c.errors.item() == 0
    with np.errstate(invalid="ignore"):
        out, lse, size = c.want()
    g = got.float().cpu().double().numpy()
    fine = np.isfinite(out)
    assert np.array_equal(np.isfinite(g), fine)
    assert np.array_equal(np.isnan(g), np.isnan(out)) and np.array_equal(g[np.isinf(out)], out[np.isinf(out)])
    tol, _ = bounds(c, lse, np.where(np.isfinite(size), size, 0))
    assert (np.abs(g - np.where(fine, out, 0)) <= tol)[fine].all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("lens", [[3, 0, 250], [126, 127, 128], [254, 121, 1]])
def test_draft_rows_do_not_see_later_ones(lens, hd, dtype):
    """NaN and infinite values and keys in the slots of later draft rows: rows that see a value get it
    back, the others nothing of it.  (Keys: a row that sees one is not a number.)"""
    K = 8
    c = Call(dtype, 3, K, 8, 2, hd, 200, lens)
    for b, n in enumerate(lens):
        c.v[b, 0, n + 2, 5] = float("nan")
        c.v[b, 0, n + 4, hd - 1] = float("inf")
        c.v[b, 0, n + 6, hd - 1] = float("-inf")
        c.v[b, 1, n + 7] = float("nan")
        c.v[b, 1, n + 1, 8] = float("-inf")
    check_rows(c)
    c = Call(dtype, 3, K, 8, 2, hd, 200, lens)
    for b, n in enumerate(lens):
        c.k[b, 0, n + 3] = float("nan")
        c.v[b, 0, n + 3] = float("nan")
    check_rows(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales_and_large_scores(dtype):
    for scale in (0.0, -0.3, 1.0, 5.0):
        c = Call(dtype, 3, 4, 8, 2, 64, 150, [3, 0, 130], scale=scale)
        if scale == 5.0:  # weights of a few slots only, references that move
            c.pk[:, ::17] *= 4
        got, lse = c.run()
        out, want, size = c.want()
        # the scores' own size enters: |s| 2^-24 (head_dim + 16) of a weight
        top = float(np.abs(want).max()) + 8
        f32 = 2 * 80 * 2.0 ** -24 * top
        tol = ((2.0 ** -7 + 2.0 ** -16 if dtype == "bf16" else 0) + f32) * size + 2.0 ** -24
        assert (np.abs(got.float().cpu().double().numpy() - out) <= tol).all(), scale
        assert np.abs(lse.cpu().double().numpy() - want).max() <= f32, scale


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_queries_and_a_larger_cache(dtype):
    B, K, nq, nkv, hd = 3, 2, 6, 2, 64
    c = Call(dtype, B, K, nq, nkv, hd, 300, [5, 140, 0], pcap=512, cap=700)
    want, wlse = c.run()
    wide = torch.full((B * K, nq * hd + 2 * nkv * hd), float("nan"), device="cuda", dtype=DT[dtype])
    view = wide[:, :nq * hd].view(B * K, nq, hd)
    view.copy_(c.q)
    c.q = view
    c.k = torch.cat([c.k, torch.full_like(c.k[:2], float("nan"))])  # request slots beyond the batch
    c.v = torch.cat([c.v, torch.full_like(c.v[:2], float("nan"))])
    got, glse = c.run()
    assert torch.equal(got, want) and torch.equal(glse, wlse)
    lse = c.lse
    c.lse.fill_(3.0)
    got, _ = c.run(out_lse=None)
    assert torch.equal(got, want) and (lse == 3.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_request_that_does_not_fit_is_left_alone(dtype):
    c = Call(dtype, 6, 4, 4, 2, 64, 100, [3, -1, 6, 7, 0, 2 ** 31 - 1][:5] + [1], cap=10)
    c.slens = ints([3, -1, 6, 7, 0, 2 ** 31 - 1])
    c.k[:, :, 4:], c.v[:, :, 4:] = 1.0, 1.0
    got, lse = c.run()
    assert c.errors.item() == pk().PEAGLE_DEV_KV_OVERFLOW
    got, lse = got.view(6, 4, 4, 64), lse.view(6, 4, 4)
    for b in (1, 3, 5):
        assert (got[b] == 7).all() and (lse[b] == 7).all()
    for b in (0, 2, 4):
        assert (got[b] != 7).all() and torch.isfinite(lse[b]).all()
    for n in (-1, 104, 2 ** 31 - 1):
        c.errors.zero_()
        c.out.fill_(5.0)
        c.plen = ints([n])
        got, _ = c.run()
        assert (got == 5).all() and c.errors.item() == pk().PEAGLE_DEV_KV_OVERFLOW


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_shared_prefix_is_the_requests_own_prefix(dtype):
    """The same rows with the prefix copied into every request: the same result within both calls'
    roundings, and for bf16 peagle_decode_attention_static's too."""
    B, K, nq, nkv, hd, P = 3, 4, 8, 2, 64, 333
    lens = [10, 0, 77]
    c = Call(dtype, B, K, nq, nkv, hd, P, lens)
    got, lse = c.run()
    whole = Call(dtype, B, K, nq, nkv, hd, 0, [P + n for n in lens], pcap=1)
    whole.q = c.q
    for mine, prefix, own in ((whole.k, c.pk, c.k), (whole.v, c.pv, c.v)):
        mine[:, :, :P] = prefix[None, :, :P]
        for b, n in enumerate(lens):
            mine[b, :, P:P + n + K] = own[b, :, :n + K]
    other, olse = whole.run()
    out, _, size = whole.want()
    tol, ltol = bounds(c, lse.cpu().double().numpy(), size)
    a, b = got.float().cpu().double().numpy(), other.float().cpu().double().numpy()
    assert (np.abs(a - b) <= 2 * tol).all() and (lse - olse).abs().max().item() <= 2 * ltol
    if dtype == "bf16":
        st = torch.zeros(B * K, nq, hd, device="cuda")
        pk().peagle_decode_attention_static(B, K, nq, nkv, hd, whole.q.float(), whole.k, whole.v, whole.k.shape[2],
                                            whole.slens, st)
        assert (np.abs(a - st.cpu().double().numpy()) <= 2 * tol).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_long_prefix(hd):
    check(Call("bf16", 2, 1, 4, 1, hd, 60001, [100, 3]))
    check(Call("bf16", 17, 4, 8, 1, hd, 5000, list(range(0, 340, 20))))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_replayed_with_other_lengths(dtype):
    c = Call(dtype, 4, 3, 8, 2, 64, 500, [7, 100, 0, 45], cap=400)
    c.k.normal_()
    c.v.normal_()
    c.pk.normal_()
    c.pv.normal_()
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk().peagle_decode_attention_shared(4, 3, c.q, c.pk, c.pv, c.plen, c.k, c.v, c.slens, c.out, c.work,
                                            out_lse=c.lse, errors=c.errors)
    for n, lens in ((500, [7, 100, 0, 45]), (3, [0, 0, 0, 0]), (129, [300, 1, 130, 397]), (0, [1, 2, 3, 4])):
        c.prefix, c.lens = n, lens
        c.plen.copy_(ints([n]))
        c.slens.copy_(ints(lens))
        c.out.fill_(9.0)
        g.replay()
        got, lse = c.out.clone(), c.lse.clone()
        c.out.fill_(8.0)
        again, l2 = c.run()
        assert torch.equal(got, again) and torch.equal(lse, l2)
        check(c)


def test_two_streams_with_a_workspace_each():
    a = Call("bf16", 5, 4, 8, 2, 64, 2000, [9, 8, 200, 1, 0], seed=3)
    b = Call("bf16", 5, 4, 8, 2, 64, 1500, [1, 300, 2, 7, 0], seed=4)
    want = [x.run()[0] for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for x, s in zip((a, b), streams):
            x.run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
