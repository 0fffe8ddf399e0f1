"""The 8-bit drafter cache on the GPU against its fp64 oracle: append and read exactly, decode
attention within bounds that follow from its roundings, and the calls together as a program
uses them (append, attend, commit, park, resume into peagle_draft, CUDA graphs, two streams)."""
import numpy as np
import pytest
import torch

import synth
from oracle import kv_quant_oracle as Q
from pe_helpers import make_ctx, oracle_draft, pk, run_draft, to_dev

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def ints(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


class Cache:
    """An 8-bit cache on the GPU, filled with random codes (NaN codes where asked) and scales."""

    def __init__(self, layers, batch, heads, capacity, hd, block, seed, spread=3, nan=0.0):
        r = np.random.default_rng(seed)
        self.block, self.shape = block, (layers, batch, heads, capacity, hd)
        sshape = (layers, batch, heads, capacity // block)
        self.t = {}
        for name in ("k", "v"):
            c = r.integers(0, 256, self.shape, dtype=np.uint8)
            c[(c & 0x7f) == 0x7f] = 0x11
            if nan:
                c[r.random(self.shape) < nan] = 0x7f
            s = np.ldexp(1.0, r.integers(-spread, spread + 1, sshape)).astype(np.float32)
            self.t[name] = torch.from_numpy(c).cuda().view(FP8)
            self.t[name + "_scale"] = torch.from_numpy(s).cuda()
        self.errors = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = pk().kv_quant_struct(self.t["k"], self.t["v"], self.t["k_scale"],
                                       self.t["v_scale"], self.errors)

    def host(self, name):
        return (self.t[name].float().cpu().double().numpy(),
                self.t[name + "_scale"].cpu().double().numpy())

    def alone(self, b):
        """Request b's part, for check_result."""
        c = Cache.__new__(Cache)
        c.block, c.t = self.block, {k: t[:, b:b + 1] for k, t in self.t.items()}
        return c

    def err(self):
        e = int(self.errors.item())
        self.errors.zero_()
        return e


def fresh(layers, batch, heads, capacity, hd, block):
    """A cache that nothing was written to yet: NaN codes and NaN scales everywhere."""
    c = Cache(layers, batch, heads, capacity, hd, block, 0)
    for name in ("k", "v"):
        c.t[name].view(torch.uint8).fill_(0x7f)
        c.t[name + "_scale"].fill_(float("nan"))
    return c


def rows_like(shape, seed, dtype, spread=4.0):
    """Rows with magnitudes over 2^+-spread and whole zero tokens, [layers, batch, n, heads, hd]."""
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape) * 2.0 ** r.uniform(-spread, spread, shape[:-1] + (1,))
    x[r.random(shape[:-1]) < 0.1] = 0.0
    return torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dtype])


def same(got, want):
    """Equal, with NaN equal to NaN."""
    return np.array_equal(got, want, equal_nan=True)


def check_append(c, lens, n, rows, before, layer=None):
    for name in ("k", "v"):
        codes, scale = before[name]
        sl = slice(None) if layer is None else slice(layer, layer + 1)
        r = rows[name].float().cpu().double().numpy()
        r = r if layer is None else r[None]
        with np.errstate(invalid="ignore"):
            wc, ws = Q.append(codes[sl], scale[sl], c.block, lens, n, r)
        codes, scale = codes.copy(), scale.copy()
        codes[sl], scale[sl] = wc, ws
        gc, gs = c.host(name)
        assert same(gs, scale), name
        assert same(gc, codes), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,block", [(64, 16), (64, 32), (64, 64), (64, 128), (128, 16),
                                      (128, 32), (128, 64), (128, 128)])
def test_append_matches_oracle(hd, block, dtype):
    m = pk()
    L, H, cap = 2, 3, 256
    # nothing committed; inside a block; at a block's end; at its first slot; up to the capacity
    lens = [0, 5, block - 1, block, cap - 9, cap, 37]
    n = [9, 9, 2, 1, 9, 0, 0]
    B = len(lens)
    c = Cache(L, B, H, cap, hd, block, 11 + hd + block, spread=12)
    rows = {k: rows_like((L, B, 9, H, hd), 5 + i + block, dtype, 12.0) for i, k in enumerate("kv")}
    before = {k: c.host(k) for k in "kv"}
    sl = ints(lens)
    m.peagle_append_kv_quant(c.kv, B, sl, ints(n), rows["k"], rows["v"], 9)
    assert c.err() == 0
    check_append(c, lens, n, rows, before)
    assert sl.tolist() == [a + b for a, b in zip(lens, n)]


def test_append_long_rows_into_an_unwritten_cache():
    """A prompt over many blocks; the cache and its scales hold NaN before."""
    m = pk()
    L, B, H, hd, cap, block = 1, 3, 2, 128, 640, 32
    c = fresh(L, B, H, cap, hd, block)
    n = [517, 1, 640]
    rows = {k: rows_like((L, B, 640, H, hd), 31 + i, "bf16") for i, k in enumerate("kv")}
    sl = ints([0, 0, 0])
    m.peagle_append_kv_quant(c.kv, B, sl, ints(n), rows["k"], rows["v"], 640)
    assert c.err() == 0 and sl.tolist() == n
    for name in ("k", "v"):
        codes, scale = c.host(name)
        for b in range(B):
            x = np.swapaxes(rows[name][:, b, :n[b]].float().cpu().double().numpy(), 1, 2)
            got = Q.values(codes, np.nan_to_num(scale, nan=1.0), block)[:, b, :, :n[b]]
            blocks = -(-n[b] // block)
            assert np.isnan(scale[:, b, :, blocks:]).all() and np.isnan(codes[:, b, :, n[b]:]).all()
            pad = np.zeros(x.shape[:2] + (blocks * block, hd))
            pad[:, :, :n[b]] = np.abs(x)
            top = pad.reshape(x.shape[:2] + (blocks, -1)).max(-1)
            assert np.array_equal(scale[:, b, :, :blocks], Q.block_scale(top))
            # half a step of e4m3, or of its smallest codes (2^-10 of the scale)
            small = np.repeat(scale[:, b, :, :blocks], block, -1)[:, :, :n[b], None] * 2.0 ** -10
            assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), small)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_special_values(dtype):
    """NaN and infinities become NaN and leave the scale alone; zero blocks get 1; values at both
    ends of the scales' range; a dropped row that had raised a scale is forgotten."""
    m = pk()
    L, B, H, hd, cap, block = 1, 6, 1, 64, 64, 16
    c = Cache(L, B, H, cap, hd, block, 3, nan=0.01)
    rows = {k: rows_like((L, B, 16, H, hd), 40 + i, dtype) for i, k in enumerate("kv")}
    for x in rows.values():
        x[0, 0, 1, 0, 3], x[0, 0, 2, 0, 5], x[0, 0, 3, 0, 60] = float("nan"), float("inf"), -float("inf")
        x[0, 1] = 0.0
        x[0, 1, 4] = -0.0
        x[0, 2] *= 1e-30
        x[0, 3] = 3.0e38
        x[0, 4] = float("nan")
    lens, n = [0, 16, 32, 0, 48, 5], [16] * 5 + [11]
    before = {k: c.host(k) for k in "kv"}
    sl = ints(lens)
    m.peagle_append_kv_quant(c.kv, B, sl, ints(n), rows["k"], rows["v"], 16, advance=False)
    assert c.err() == 0 and sl.tolist() == lens
    check_append(c, lens, n, rows, before)
    assert (c.t["k_scale"][0, 1, 0, 1] == 1.0) and (c.t["k_scale"][0, 4, 0, 3] == 1.0)
    # request 5's rows are dropped; a quieter row takes their place and the scale shrinks again
    before = {k: c.host(k) for k in "kv"}
    quiet = {k: x * 2.0 ** -9 for k, x in rows.items()}
    m.peagle_append_kv_quant(c.kv, B, sl, ints([0] * 5 + [1]), quiet["k"], quiet["v"], 16)
    check_append(c, lens, [0] * 5 + [1], quiet, before)


def test_append_strides_layers_and_counts():
    """Rows out of a fused projection and out of a peagle_kv buffer; one layer; n_extra; n_commit
    absent; bad requests left alone."""
    m = pk()
    L, B, H, hd, cap, block = 3, 4, 2, 64, 64, 32
    c = Cache(L, B, H, cap, hd, block, 8)
    fused = rows_like((B, 5, 3 * H, hd), 50, "bf16")  # queries | keys | values of one layer
    rows = {"k": fused[:, :, H:2 * H], "v": fused[:, :, 2 * H:]}
    before = {k: c.host(k) for k in "kv"}
    lens = [3, 0, 30, 59]
    m.peagle_append_kv_quant(c.kv, B, ints(lens), ints([1, 2, 3, 4]), rows["k"], rows["v"], 5,
                             layer=1, n_extra=1, advance=False)
    assert c.err() == 0
    check_append(c, lens, [2, 3, 4, 5], rows, before, layer=1)

    kv16 = rows_like((2, L, B, H, cap, hd), 51, "bf16")  # k and v as peagle_kv holds them
    rows = {"k": kv16[0].transpose(2, 3), "v": kv16[1].transpose(2, 3)}
    before = {k: c.host(k) for k in "kv"}
    m.peagle_append_kv_quant(c.kv, B, ints([0] * B), None, rows["k"], rows["v"], 7, n_extra=7)
    check_append(c, [0] * B, [7] * B, rows, before)
    # fewer requests than the cache holds; rows in reverse order of tokens and of requests
    back = {k: x.flip(1).contiguous() for k, x in rows.items()}
    before = {k: c.host(k) for k in "kv"}
    m.peagle_append_kv_quant(c.kv, 2, ints([9, 9]), ints([4, 6]), back["k"][:, :2], back["v"][:, :2], 6)
    check_append(c, [9, 9], [4, 6], {k: x[:, :2] for k, x in back.items()}, before)

    before = {k: c.host(k) for k in "kv"}
    big = 2 ** 31 - 1
    for lens, n, extra, bits in (([0, 62, 0, 0], [1, 3, 0, 0], 0, m.PEAGLE_DEV_KV_OVERFLOW),
                                 ([0, -1, 0, 0], [1, 1, 0, 0], 0, m.PEAGLE_DEV_KV_OVERFLOW),
                                 ([0, 0, 0, big], [1, 0, 0, 1], 0, m.PEAGLE_DEV_KV_OVERFLOW),
                                 ([0, 0, 0, 0], [1, 8, -1, big], 0, m.PEAGLE_DEV_BAD_COMMIT),
                                 ([0, 0, 0, 0], [0, big, -big - 1, 0], 1, m.PEAGLE_DEV_BAD_COMMIT)):
        sl = ints(lens)
        m.peagle_append_kv_quant(c.kv, B, sl, ints(n), rows["k"], rows["v"], 7, n_extra=extra)
        assert c.err() == bits, (lens, n)
        ok = [0 <= x + extra <= 7 and 0 <= a <= cap - (x + extra) for a, x in zip(lens, n)]
        assert sl.tolist() == [a + (x + extra if o else 0) for a, x, o in zip(lens, n, ok)]
        check_append(c, [a if o else 0 for a, o in zip(lens, ok)],
                     [x + extra if o else 0 for x, o in zip(n, ok)], rows, before)
        before = {k: c.host(k) for k in "kv"}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
def test_read_matches_codes_times_scales(hd, block, dtype):
    m = pk()
    L, B, H, cap = 2, 5, 3, 512
    c = Cache(L, B, H, cap, hd, block, 60, spread=20, nan=0.001)
    # a scale that is no power of two is rounded once
    c.t["v_scale"][0, 0] = 0.1
    starts, n = [0, 17, 511, cap, 130], [300, 129, 1, 0, 70]
    for layer in (-1, 1):
        sh = (B, H, 301, hd) if layer >= 0 else (L, B, H, 301, hd)
        out = {k: torch.full(sh, -7.0, dtype=DT[dtype], device="cuda") for k in "kv"}
        m.peagle_read_kv_quant(c.kv, B, ints(n), out["k"].transpose(-3, -2),
                               out["v"].transpose(-3, -2), 300, layer=layer, starts=ints(starts))
        assert c.err() == 0
        for name in "kv":
            codes, scale = c.host(name)
            want = torch.from_numpy(codes).float() * torch.from_numpy(
                np.repeat(scale, block, -1)[..., None]).float()
            want = want.to(DT[dtype]).float().numpy()
            want = want if layer < 0 else want[layer:layer + 1]
            got = out[name].float().cpu().numpy()
            got = got if layer < 0 else got[None]
            for b in range(B):
                assert same(got[:, b, :, :n[b]], want[:, b, :, starts[b]:starts[b] + n[b]])
                assert (got[:, b, :, n[b]:] == -7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_ragged_calls_equal_their_layers(dtype):
    """Calls so large that a CTA takes several parts of its request's rows, against calls for one
    layer, which are not."""
    m = pk()
    L, B, H, hd, cap, block = 4, 20, 8, 64, 2048, 16
    c, one = fresh(L, B, H, cap, hd, block), fresh(L, B, H, cap, hd, block)
    n = [2000, 0, 1, 15, 16, 17, 33, 1999, 64, 500, 31, 1024, 1, 0, 1500, 100, 48, 49, 2000, 700]
    at = [48, 5, 2047, 0, 16, 3, 31, 0, 1, 17, 0, 1000, 8, 9, 0, 100, 7, 47, 33, 1]
    rows = [torch.randn(L, B, 2000, H, hd, device="cuda",
                        generator=torch.Generator("cuda").manual_seed(i)).to(DT[dtype]) for i in (1, 2)]
    sl, so = ints(at), ints(at)
    m.peagle_append_kv_quant(c.kv, B, sl, ints(n), *rows, 2000)
    for layer in range(L):
        m.peagle_append_kv_quant(one.kv, B, so, ints(n), rows[0][layer], rows[1][layer], 2000,
                                 layer=layer, advance=layer == L - 1)
    assert c.err() == 0 and one.err() == 0 and torch.equal(sl, so)
    for name in c.t:
        assert torch.equal(c.t[name].view(torch.uint8), one.t[name].view(torch.uint8)), name
    out = torch.full((2, 2, L, B, 2000, H, hd), -7.0, dtype=DT[dtype], device="cuda")
    m.peagle_read_kv_quant(c.kv, B, ints(n), out[0, 0], out[0, 1], 2000, starts=ints(at))
    for layer in range(L):
        m.peagle_read_kv_quant(c.kv, B, ints(n), out[1, 0, layer], out[1, 1, layer], 2000,
                               layer=layer, starts=ints(at))
    assert c.err() == 0 and torch.equal(out[0], out[1])
    for b in range(B):
        assert (out[0, :, :, b, n[b]:] == -7.0).all()
        assert not n[b] or (out[0, :, :, b, :n[b]] != -7.0).any(-1).all()


def test_read_counts_out_of_range():
    m = pk()
    c = Cache(1, 3, 2, 64, 64, 16, 61)
    out = torch.full((2, 1, 3, 10, 2, 64), -7.0, device="cuda")
    for starts, n, bits in (([0, 0, 0], [4, -1, 11], m.PEAGLE_DEV_BAD_COMMIT),
                            ([0, 60, -1], [4, 5, 1], m.PEAGLE_DEV_KV_OVERFLOW)):
        m.peagle_read_kv_quant(c.kv, 3, ints(n), out[0], out[1], 10, starts=ints(starts))
        assert c.err() == bits
        assert (out[:, :, 0, :4] != -7.0).any(-1).all()
        assert (out[:, :, 1:] == -7.0).all() and (out[:, :, 0, 4:] == -7.0).all()
    with pytest.raises(m.PeagleError):  # rows that overlap
        one = out[:, :, :, :1].expand(2, 1, 3, 10, 2, 64)
        m.peagle_read_kv_quant(c.kv, 3, ints([1, 1, 1]), one[0], one[1], 10)


# ---- attention ----------------------------------------------------------------------

def bounds(q, kval, vval, vscale_max, lens, K, causal, window, scale, out, lse, absolute, dtype):
    """Largest errors that the documented arithmetic allows, per output element and per lse.

    u = 2^-24 is half an fp32 step.  A score is a product of hd terms summed in fp32 in any
    order: (hd + 8) u S with S = scale sum |q k|; fp32 queries come as two 11-bit parts, which
    drop 2^-22 of an element, or of 2^-2 of the row's largest where an element is that small:
    2^-22 S + 2^-24 scale max|q| sum |k|.  A score's error d moves the weights by 2 d relative
    (numerator and sum).  The exponential's argument carries u of its size (|x| < 2^8 before a
    weight vanishes: 2^-16 absolute is 2^8 u) and the SFU 2^-21.  Weights are rounded to f16's 11
    bits in the numerator and not in the sum: consecutive values with e = 2^k <= w < 2^(k+1) are
    2^-10 e apart, so half a step is 2^-11 e <= 2^-11 w (one slot seen alone gets all of it: its
    result is v round(w) / w).  fp32's second part holds the rest, at most 2^-11 w, to 11 bits
    again: 2^-22 or, below f16's normal values, to half
    of 2^-24 where the largest weight x value scale of the row is at least 2^-4 (2^13 for fp32):
    n 2^-21 448 s over all slots (2^-38), s the largest value scale.  Sums over n slots:
    (n + 64) u.  Then half a step of the output's type."""
    f32 = dtype == "f32"
    u = 2.0 ** -24
    BK, nq, hd = q.shape
    G = nq // kval.shape[1]
    to, tl = np.zeros_like(out), np.zeros_like(lse)
    for r in range(BK):
        b, j = divmod(r, K)
        begin, end = Q.span(int(lens[b]), j, causal, window)
        n = max(0, end - begin)
        if not n:
            continue
        for h in range(nq):
            ak = np.abs(kval[b, h // G, begin:end])
            S = abs(scale) * (ak @ np.abs(q[r, h])).max()
            d = (hd + 8) * u * S
            if f32:
                d += 2.0 ** -22 * S + u * abs(scale) * np.abs(q[r, h]).max() * ak.sum(-1).max()
            d += 2.0 ** -15 + 2.0 ** -21 + 4 * u * S
            w, tiny = (2.0 ** -22, 2.0 ** -38) if f32 else (2.0 ** -11, 2.0 ** -21)
            to[r, h] = absolute[r, h] * (2 * d + w + 2 * (n + 64) * u) + \
                n * tiny * 448.0 * vscale_max[b, h // G]
            tl[r, h] = d + (n + 64) * u + 4 * u * abs(lse[r, h])
    half = u if f32 else 2.0 ** -8
    return to * (1 + half) + half * np.abs(out), tl


def attend(c, layer, q, lens, K, causal=True, window=0, scale=None, stream=None, work=None):
    m = pk()
    B, nq = len(lens), q.shape[1]
    out = torch.full(q.shape, -7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], -7.0, device="cuda")
    if work is None:
        n = m.peagle_decode_attention_quant_workspace(c.kv, B, K, nq)
        work = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # NaN wherever it is read
    m.peagle_decode_attention_quant(c.kv, layer, B, K, nq, q, ints(lens), out, work, out_lse=lse,
                                    causal=causal, window=window, scale=scale)
    return out, lse


def check_result(c, layer, q, lens, K, causal, window, scale, out, lse):
    dtype = "f32" if q.dtype == torch.float32 else "bf16"
    q64 = q.double().cpu().numpy()
    B = len(lens)
    (kc, ks), (vc, vs) = c.host("k"), c.host("v")
    kval, vval = (Q.values(x[layer, :B], y[layer, :B], c.block) for x, y in ((kc, ks), (vc, vs)))
    sc = q.shape[2] ** -0.5 if scale is None else scale
    want, wl, ab = Q.attention(q64, kval, vval, lens, K, causal, window, sc)
    to, tl = bounds(q64, kval, vval, vs[layer].max(-1), lens, K, causal, window, sc, want, wl, ab,
                    dtype)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    none = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), none) and not got[none].any()
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / np.where(to > 0, to, 1))
    assert worst <= 1, f"out: {worst:.3f} of the bound"
    if not none.all():
        worst = np.max(np.abs(gl[~none] - wl[~none]) / tl[~none])
        assert worst <= 1, f"lse: {worst:.3f} of the bound"


def check_attention(c, layer, q, lens, K, causal=True, window=0, scale=None):
    out, lse = attend(c, layer, q, lens, K, causal, window, scale)
    assert c.err() == 0
    check_result(c, layer, q, lens, K, causal, window, scale, out, lse)
    return out, lse


def queries(B, K, nq, hd, dtype, seed, size=1.0):
    r = np.random.default_rng(seed)
    # codes are up to 448 of their scale: queries that keep the scores within some tens
    x = r.standard_normal((B * K, nq, hd)) * 2.0 ** r.uniform(-3, 0, (B * K, nq, 1)) * size / 100
    return torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dtype])


# (q heads, kv heads, head_dim, K, block): 1 to 128 query rows a kv head, whole and odd
SHAPES = [(1, 1, 64, 1, 16), (2, 2, 128, 1, 32), (4, 2, 64, 4, 32), (8, 1, 128, 1, 64),
          (9, 3, 64, 3, 128), (8, 2, 128, 5, 16), (14, 2, 64, 3, 64), (16, 2, 64, 4, 32),
          (8, 2, 128, 8, 64), (16, 2, 128, 5, 128), (16, 1, 64, 3, 32), (16, 2, 64, 8, 16),
          (8, 1, 128, 8, 32), (16, 1, 128, 7, 32), (32, 2, 64, 8, 64), (16, 1, 128, 8, 16),
          (16, 2, 64, 13, 32), (7, 1, 128, 16, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv,hd,K,block", SHAPES)
def test_attention_matches_oracle(nq, nkv, hd, K, block, dtype):
    # empty, one slot, around 16 and the block, several CTAs' shares
    lens = [0, 1, 15, 16, 33, block - 1, 517]
    B = len(lens)
    cap = (517 + K + block - 1) // block * block
    c = Cache(2, B, nkv, cap, hd, block, nq + hd + K, spread=4)
    q = queries(B, K, nq, hd, dtype, K + nq)
    check_attention(c, 1, q, lens, K)
    check_attention(c, 0, q, lens, K, causal=False)
    check_attention(c, 0, q, lens, K, window=max(2, K // 2))
    check_attention(c, 1, q, lens, K, causal=False, window=100)
    check_attention(c, 1, q, lens, K, scale=-0.05)


# more than 48 (head_dim 128: 32) query rows a kv head and enough slots that the tcgen05 kernel runs:
# whole and odd row counts, one and two parts of them, one and two kv heads
MANY_ROWS = [(8, 1, 64, 7, 16, 28672), (16, 1, 64, 4, 32, 28672), (32, 2, 64, 4, 64, 14336),
             (7, 1, 64, 16, 128, 14336), (11, 1, 128, 3, 16, 28672), (8, 1, 128, 5, 32, 28672),
             (16, 2, 128, 8, 64, 14336), (9, 1, 128, 11, 128, 14336), (16, 1, 128, 8, 16, 14336)]


@pytest.mark.parametrize("nq,nkv,hd,K,block,cap", MANY_ROWS)
def test_attention_many_rows(nq, nkv, hd, K, block, cap):
    # around the kernel's tiles of 128 slots
    lens = [0, 1, 120, 128, 129, 517, 383]
    c = Cache(1, len(lens), nkv, cap, hd, block, nq + hd + K, spread=4)
    q = queries(len(lens), K, nq, hd, "bf16", K + nq)
    check_attention(c, 0, q, lens, K)
    check_attention(c, 0, q, lens, K, causal=False)
    check_attention(c, 0, q, lens, K, causal=False, scale=-0.05)
    # (a window keeps the slots that a call sees few; at 28,088 and more the tcgen05 kernel runs)
    check_attention(c, 0, q, lens, K, window=max(2, K // 2))
    # the end of the capacity
    lens = [cap - K, cap - 100, cap - 129 - K, 5, 5, 5, 5]
    check_attention(c, 0, q, lens, K)


@pytest.mark.parametrize("hd,G,K", [(64, 16, 4), (128, 8, 5), (128, 16, 8)])
def test_attention_many_rows_long_and_many(hd, G, K):
    """Heads over several CTAs beside short ones; more heads than CTAs; a window in long contexts."""
    lens = [16000, 3, 9000]
    c = Cache(1, 3, 4, 16512, hd, 32, 5, spread=2)
    q = queries(3, K, 4 * G, hd, "bf16", 77)
    check_attention(c, 0, q, lens, K)
    lens = [int(x) for x in np.random.default_rng(9).integers(0, 300, 300)]
    lens[7] = 4000
    c = Cache(1, 300, 1, 4096, hd, 16, 6, spread=2)
    q = queries(300, K, G, hd, "bf16", 78)
    check_attention(c, 0, q, lens, K)
    check_attention(c, 0, q, lens, K, window=1000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,G,K", [(64, 1, 1), (64, 4, 3), (64, 8, 8), (128, 8, 1), (128, 4, 5),
                                    (128, 16, 8)])
@pytest.mark.parametrize("heads", [1, 3, 7, 20])
def test_attention_heads_shared_by_clusters(hd, G, K, heads, dtype):
    """Capacities at which several CTAs share a head in one launch: 8, 4, 2 and 1 of them, shares
    without a tile, requests that are empty or do not fit beside others of the same cluster."""
    m = pk()
    lens = [2040, 0, 1, 33, 300]
    c = Cache(1, 5, heads, 2048, hd, 32, heads + hd, spread=2)
    q = queries(5, K, heads * G, hd, dtype, 80)
    check_attention(c, 0, q, lens, K)
    check_attention(c, 0, q, [5, 6, 2048, 640, 31], K, causal=False)
    check_attention(c, 0, q, [1111, 1999, 2, 640, 0], K, window=100)
    bad = [5, -1, 2049, 640, 700]
    out, lse = attend(c, 0, q, bad, K)
    assert c.err() == m.PEAGLE_DEV_KV_OVERFLOW
    for b in range(5):
        rows = slice(b * K, (b + 1) * K)
        if b in (1, 2):
            assert (out[rows] == -7.0).all() and (lse[rows] == -7.0).all()
        else:
            check_result(c.alone(b), 0, q[rows], [bad[b]], K, True, 0, None, out[rows], lse[rows])


# one launch, two, and the tcgen05 kernel
@pytest.mark.parametrize("nq,cap", [(8, 160), (8, 2048), (32, 98304)])
def test_attention_windows_that_reach_every_slot(nq, cap):
    """The largest window that leaves a slot out, the smallest that leaves none, and the largest."""
    K = 7
    c = Cache(1, 2, 2, cap, 64, 32, 8, spread=2)
    q = queries(2, K, nq, 64, "bf16", 79)
    lens = [cap - K, 130]
    for causal in (True, False):
        out, lse = check_attention(c, 0, q, lens, K, causal=causal)
        for window in (cap, cap + K, cap + K + 1, 2 ** 31 - 1):
            got = check_attention(c, 0, q, lens, K, causal=causal, window=window)
            assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        check_attention(c, 0, q, lens, K, causal=causal, window=cap - 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv,hd,K", [(8, 1, 64, 8), (4, 1, 128, 1), (16, 1, 128, 8)])
def test_attention_long_context(nq, nkv, hd, K, dtype):
    """Two requests split over every SM, one short one beside them."""
    lens = [6011, 3, 9000]
    c = Cache(1, 3, nkv, 9024, hd, 32, 5, spread=2)
    q = queries(3, K, nq, hd, dtype, 77)
    check_attention(c, 0, q, lens, K)
    check_attention(c, 0, q, lens, K, window=4000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,G,K", [(64, 2, 4), (128, 1, 3), (64, 8, 8), (128, 4, 16)])
def test_attention_many_requests(hd, G, K, dtype):
    """More (request, kv head) pairs than CTAs, ragged."""
    lens = [int(x) for x in np.random.default_rng(9).integers(0, 180, 300)]
    c = Cache(1, 300, 2, 208, hd, 16, 6, spread=2)
    check_attention(c, 0, queries(300, K, 2 * G, hd, dtype, 78), lens, K)


@pytest.mark.parametrize("nq,hd,K,cap,dtype", [
    (4, 64, 4, 160, "bf16"), (4, 64, 4, 160, "f32"), (2, 128, 8, 160, "bf16"),
    (2, 128, 8, 160, "f32"), (16, 64, 8, 160, "bf16"), (16, 64, 8, 160, "f32"),
    # tcgen05
    (16, 64, 8, 24576, "bf16"), (8, 128, 5, 49152, "bf16"), (12, 128, 7, 24576, "bf16")])
def test_attention_unseen_slots_never_matter(nq, hd, K, cap, dtype):
    """Every slot that no row sees, and every scale of such blocks, is NaN; slots that only some
    rows see (the draft block, the window's edge) hold NaN for the rows that do not see them."""
    m = pk()
    lens = [0, 7, 40, 129]
    B, block = len(lens), 16
    c = Cache(1, B, 1, cap, hd, block, 21)
    q = queries(B, K, nq, hd, dtype, 22)
    wide = cap // 2  # the rows' last slots again, and one window that reaches all of them
    for causal, window in ((True, 0), (False, 0), (True, 9), (True, 50), (False, 30), (True, wide)):
        want, wl = attend(c, 0, q, lens, K, causal, window)
        keep = {n: t.clone() for n, t in c.t.items()}
        for b, n in enumerate(lens):
            seen = np.zeros(cap, bool)
            for j in range(K):
                lo, hi = Q.span(n, j, causal, window)
                seen[lo:max(lo, hi)] = True
            t = torch.from_numpy(~seen).cuda()
            for name in ("k", "v"):
                c.t[name].view(torch.uint8)[0, b, :, t] = 0x7f
                blk = torch.from_numpy(~seen.reshape(-1, block).any(-1)).cuda()
                c.t[name + "_scale"][0, b, :, blk] = float("nan")
        got, gl = attend(c, 0, q, lens, K, causal, window)
        assert torch.equal(got, want) and torch.equal(gl, wl), (causal, window)
        # the last draft row's own slot: NaN in it reaches that row alone
        if causal and not window:
            for name in ("k", "v"):
                for b, n in enumerate(lens):
                    c.t[name].view(torch.uint8)[0, b, :, n + K - 1, 5] = 0xff
                got, gl = attend(c, 0, q, lens, K, causal, window)
                g, w = got.view(B, K, nq, hd), want.view(B, K, nq, hd)
                assert torch.equal(g[:, :-1], w[:, :-1])
                if name == "v":
                    assert torch.isnan(g[:, -1, :, 5]).all() and torch.isfinite(gl).all()
                    rest = [d for d in range(hd) if d != 5]
                    assert torch.equal(g[:, -1, :, rest], w[:, -1, :, rest])
                else:
                    assert torch.isnan(g[:, -1]).all()
                    assert torch.isnan(gl.view(B, K, nq)[:, -1]).all()
                for n_, t in keep.items():
                    c.t[n_].copy_(t)
        # the window's first row alone sees its first slot
        if causal and window == 50:
            c.t["v"].view(torch.uint8)[0, 3, :, 129 - window + 1, 7] = 0x7f
            got, gl = attend(c, 0, q, lens, K, causal, window)
            g, w = got.view(B, K, nq, hd), want.view(B, K, nq, hd)
            assert torch.equal(g[3, 1:], w[3, 1:]) and torch.equal(g[:3], w[:3])
            assert torch.isnan(g[3, 0, :, 7]).all() and torch.isfinite(g[3, 0, :, 8:]).all()
        for n_, t in keep.items():
            c.t[n_].copy_(t)


@pytest.mark.parametrize("nq,cap,dtype", [(4, 416, "bf16"), (4, 416, "f32"), (32, 98304, "bf16")])
def test_attention_scales_far_apart(nq, cap, dtype):
    """Blocks whose scales differ by 2^40, zero blocks among them, and any scale, not only powers
    of two; sharp and flat rows; large and tiny queries."""
    lens, K, hd, block = [400, 90], 2, 64, 16
    for seed, size in ((1, 1.0), (2, 30.0), (3, 1e-6)):
        c = Cache(1, 2, 1, cap, hd, block, seed, spread=0)
        r = np.random.default_rng(seed)
        s = 2.0 ** r.uniform(-20, 20, (1, 2, 1, cap // block))
        c.t["v_scale"].copy_(torch.from_numpy(s.astype(np.float32)))
        c.t["k_scale"].copy_(torch.from_numpy((2.0 ** r.uniform(-1, 1, s.shape)).astype(np.float32)))
        c.t["v"].view(torch.uint8)[0, :, :, 32:48] = 0
        check_attention(c, 0, queries(2, K, nq, hd, dtype, seed, size), lens, K)


@pytest.mark.parametrize("nq,cap", [(2, 64), (32, 98304)])
def test_attention_queries_that_are_not_finite(nq, cap):
    lens, K, hd = [50, 7], 2, 64
    c = Cache(1, 2, 1, cap, hd, 32, 4)
    for dtype in ("bf16", "f32"):
        q = queries(2, K, nq, hd, dtype, 5)
        want, _ = attend(c, 0, q, lens, K)
        for bad in (float("nan"), float("inf"), -float("inf")):
            p = q.clone()
            p[1, 0, 9] = bad
            got, lse = attend(c, 0, p, lens, K)
            ok = torch.ones(4, nq, dtype=torch.bool, device="cuda")
            ok[1, 0] = False
            assert torch.equal(got[ok], want[ok]) and torch.isfinite(lse[ok]).all()
            assert torch.isnan(got[1, 0]).all()
        # a row of zeros weighs every slot alike
        p = torch.zeros_like(q)
        check_attention(c, 0, p, lens, K)


@pytest.mark.parametrize("nq,cap", [(4, 96), (32, 19680)])
def test_attention_requests_out_of_range_and_strided_queries(nq, cap):
    m = pk()
    K, hd = 3, 128
    c = Cache(1, 5, 2, cap, hd, 32, 30)
    fused = queries(5, K, 2 * nq, hd, "bf16", 31)
    q = fused[:, :nq]  # rows of a fused projection
    lens = [5, -1, cap - K, cap - K + 1, 2 ** 31 - 1]
    out, lse = attend(c, 0, q, lens, K)
    assert c.err() == m.PEAGLE_DEV_KV_OVERFLOW
    for b, n in ((0, 5), (2, cap - K)):
        one = slice(b * K, (b + 1) * K)
        check_result(c.alone(b), 0, q[one], [n], K, True, 0, None, out[one], lse[one])
    for b in (1, 3, 4):
        assert (out[b * K:(b + 1) * K] == -7.0).all() and (lse[b * K:(b + 1) * K] == -7.0).all()
    out, _ = attend(c, 0, q, [5, 1, 2, cap - K + 1, cap], K, causal=False)  # the prefix alone fits
    assert c.err() == 0 and (out != -7.0).any(-1).all()
    # without lse the output is the same, and so it is with contiguous queries
    lens = [5, 0, cap - K]
    ref, _ = attend(c, 0, q[:3 * K].contiguous(), lens, K)
    o2 = torch.empty(3 * K, nq, hd, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(m.peagle_decode_attention_quant_workspace(c.kv, 3, K, nq), dtype=torch.uint8,
                    device="cuda")
    m.peagle_decode_attention_quant(c.kv, 0, 3, K, nq, q[:3 * K], ints(lens), o2, w)
    assert torch.equal(o2, ref)


def test_offsets_beyond_32_bits():
    """A cache whose codes pass 4 GB in one layer: the last head of the last request is written,
    attended and read back."""
    m = pk()
    B, H, hd, block = 2, 2, 128, 128
    cap = 9 * (1 << 20)
    c = Cache.__new__(Cache)
    c.block, c.errors = block, torch.zeros(1, dtype=torch.int32, device="cuda")
    c.t = {}
    for name in ("k", "v"):
        c.t[name] = torch.zeros(1, B, H, cap, hd, dtype=torch.uint8, device="cuda").view(FP8)
        c.t[name + "_scale"] = torch.ones(1, B, H, cap // block, device="cuda")
    assert c.t["k"].numel() > 1 << 32
    c.kv = m.kv_quant_struct(c.t["k"], c.t["v"], c.t["k_scale"], c.t["v_scale"], c.errors)
    at = cap - 300
    rows = {k: rows_like((1, B, 300, H, hd), 70 + i, "bf16", 1.0) for i, k in enumerate("kv")}
    m.peagle_append_kv_quant(c.kv, B, ints([0, at]), ints([0, 300]), rows["k"], rows["v"], 300)
    out = torch.zeros(2, 1, B, 300, H, hd, device="cuda")
    m.peagle_read_kv_quant(c.kv, B, ints([0, 300]), out[0], out[1], 300, starts=ints([0, at]))
    for i, k in enumerate("kv"):
        x = rows[k][0, 1].float()
        assert ((out[i, 0, 1] - x).abs() <= x.abs().amax() * 2.0 ** -4).all()
        assert out[i, 0, 1].abs().sum() > 0
    q = queries(B, 1, H, hd, "bf16", 71, 100.0)
    got, lse = attend(c, 0, q, [1, cap], 1, causal=False, window=301)
    assert c.err() == 0
    k, v = out[0, 0, 1].double(), out[1, 0, 1].double()  # [300, H, hd]
    s = torch.einsum("hd,thd->ht", q[1].double(), k) * hd ** -0.5
    want = torch.einsum("ht,thd->hd", s.softmax(-1), v)
    assert (got[1].double() - want).abs().max() <= 2.0 ** -7 * v.abs().max()
    assert (lse[1].double() - torch.logsumexp(s, -1)).abs().max() <= 1e-4


# ---- together, as a program uses them ------------------------------------------------

def test_decode_rounds_of_append_attend_commit():
    """Several rounds: the draft block's K/V of each layer written, attended by the block, some of
    the rows committed and the rest dropped; one layer at a time as a drafter runs them."""
    m = pk()
    L, B, H, nq, hd, K, block, cap = 2, 3, 2, 8, 64, 4, 16, 96
    c = fresh(L, B, H, cap, hd, block)
    ref = {k: (np.zeros((L, B, H, cap, hd)), np.ones((L, B, H, cap // block))) for k in "kv"}
    lens = [0, 11, 30]
    prompt = {k: rows_like((L, B, 30, H, hd), 80 + i, "bf16", 1.0) for i, k in enumerate("kv")}
    sl, n = ints([0] * B), ints(lens)
    m.peagle_append_kv_quant(c.kv, B, sl, n, prompt["k"], prompt["v"], 30)
    host = lambda t: t.float().cpu().double().numpy()  # noqa: E731
    for k in "kv":
        ref[k] = Q.append(*ref[k], block, [0] * B, lens, host(prompt[k]))
    work = torch.empty(m.peagle_decode_attention_quant_workspace(c.kv, B, K, nq), dtype=torch.uint8,
                       device="cuda")
    for step in range(6):
        rows = {k: rows_like((L, B, K, H, hd), 90 + 2 * step + i, "bf16", 3.0)
                for i, k in enumerate("kv")}
        q = queries(B, K, nq, hd, "bf16", step, 10.0)
        accepted = [(step + b) % (K + 1) for b in range(B)]
        for layer in range(L):
            m.peagle_append_kv_quant(c.kv, B, sl, None, rows["k"][layer], rows["v"][layer], K,
                                     layer=layer, n_extra=K, advance=False)
        for k in "kv":
            ref[k] = Q.append(*ref[k], block, lens, [K] * B, host(rows[k]))
        for layer in range(L):
            out = torch.empty_like(q)
            m.peagle_decode_attention_quant(c.kv, layer, B, K, nq, q, sl, out, work)
            kval, vval = (Q.values(ref[k][0][layer], ref[k][1][layer], block) for k in "kv")
            q64 = q.double().cpu().numpy()
            want, wl, ab = Q.attention(q64, kval, vval, lens, K)
            to, _ = bounds(q64, kval, vval, ref["v"][1][layer].max(-1), lens, K, True, 0,
                           hd ** -0.5, want, wl, ab, "bf16")
            assert (np.abs(out.double().cpu().numpy() - want) <= to).all()
        # the commit appends the accepted rows once more: the dropped ones leave the scales
        m.peagle_append_kv_quant(c.kv, B, sl, ints(accepted), rows["k"], rows["v"], K)
        for k in "kv":
            ref[k] = Q.append(*ref[k], block, lens, accepted, host(rows[k]))
        lens = [a + b for a, b in zip(lens, accepted)]
        assert sl.tolist() == lens and c.err() == 0
    for k in "kv":
        codes, scale = c.host(k)
        for b in range(B):
            got = Q.values(codes, np.nan_to_num(scale, nan=0.0), block)[:, b, :, :lens[b]]
            assert np.array_equal(got, Q.values(*ref[k], block)[:, b, :, :lens[b]])


def test_parked_request_resumes_the_draft_pass():
    """A request's 16-bit cache is parked in 8 bits and read back into a peagle_kv buffer; the
    draft pass on it equals the oracle's on the rounded cache."""
    m = pk()
    dims = synth.shrink(synth.DIMS_TINY, dtype="bf16", n_layers=2)
    K, B, block = 4, 2, 32
    wl = synth.Workload("parked", dims, B, K, (70, 33))
    w, inp = synth.make_weights(dims, 4), synth.make_decode_inputs(wl, 5)
    cap = inp["capacity"]
    d = to_dev(inp)
    cap8 = (cap + block - 1) // block * block
    c = fresh(dims.n_layers, B, dims.n_kv_heads, cap8, dims.head_dim, block)
    at = ints([0, 0])
    m.peagle_append_kv_quant(c.kv, B, at, d["sl"], d["ck"].transpose(2, 3), d["cv"].transpose(2, 3), cap)
    assert torch.equal(at, d["sl"])
    back = {k: torch.zeros_like(d["c" + k]) for k in "kv"}
    m.peagle_read_kv_quant(c.kv, B, d["sl"], back["k"].transpose(2, 3), back["v"].transpose(2, 3), cap)
    assert c.err() == 0
    for k in "kv":
        for b, n in enumerate((70, 33)):
            x, y = d["c" + k][:, b, :, :n].float(), back[k][:, b, :, :n].float()
            assert ((x - y).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -17 * x.abs().max()).all()
            assert not torch.equal(x, y)
    rounded = dict(inp, cache_k=back["k"].cpu(), cache_v=back["v"].cpu())
    ctx = make_ctx(dims, w, B, K, cap)
    d["ck"], d["cv"] = back["k"], back["v"]
    toks, lg, _ = run_draft(ctx, dims, rounded, K, d)
    ctx.close()
    ref = oracle_draft(dims, w, rounded, K)
    assert float(np.max(np.abs(lg - ref.logits))) <= 2e-2
    ok = ref.margin > 1e-2
    assert np.array_equal(toks[ok], ref.tokens[ok])


# one launch, clusters of 8 CTAs, two launches, the tcgen05 kernel
@pytest.mark.parametrize("nq,cap,window", [(8, 160, 70), (8, 2048, 0), (8, 12288, 0), (16, 49152, 0)])
def test_captured_round_replays_on_new_inputs(nq, cap, window):
    """append + attention + commit in one CUDA graph, replayed while lengths advance, beside an
    eager call with its own workspace on another stream."""
    m = pk()
    L, B, H, hd, K, block = 1, 2, 2, 128, 5, 32
    c, e = fresh(L, B, H, cap, hd, block), fresh(L, B, H, cap, hd, block)
    rows = torch.zeros(2, L, B, K, H, hd, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B * K, nq, hd, dtype=torch.bfloat16, device="cuda")
    out, n = torch.zeros_like(q), torch.zeros(B, dtype=torch.int32, device="cuda")
    sl = ints([0, 0])
    size = m.peagle_decode_attention_quant_workspace(c.kv, B, K, nq)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step(c, sl, rows, q, n, out, work):
        m.peagle_append_kv_quant(c.kv, B, sl, None, rows[0], rows[1], K, n_extra=K, advance=False)
        m.peagle_decode_attention_quant(c.kv, 0, B, K, nq, q, sl, out, work, window=window)
        m.peagle_append_kv_quant(c.kv, B, sl, n, rows[0], rows[1], K)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c, sl, rows, q, n, out, work)
    torch.cuda.current_stream().wait_stream(side)
    sl.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c, sl, rows, q, n, out, work)
    esl, eout = ints([0, 0]), torch.zeros_like(q)
    ework = torch.empty(size, dtype=torch.uint8, device="cuda")
    for i in range(20):
        rows.copy_(rows_like(tuple(rows.shape), 200 + i, "bf16", 2.0))
        q.copy_(queries(B, K, nq, hd, "bf16", 300 + i, 5.0))
        n.copy_(ints([i % (K + 1), K]))
        side.wait_stream(torch.cuda.current_stream())
        g.replay()
        with torch.cuda.stream(side):
            step(e, esl, rows, q, n, eout, ework)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, eout) and torch.equal(sl, esl)
    assert sl.tolist() == [sum(i % (K + 1) for i in range(20)), 20 * K]
    for k in c.t:
        assert torch.equal(c.t[k].view(torch.uint8), e.t[k].view(torch.uint8))
    assert c.err() == 0 and e.err() == 0
