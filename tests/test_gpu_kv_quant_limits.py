"""Decode attention over the 8-bit cache where its arithmetic is at its limits, against the fp64
oracle with a tolerance taken from what each row sees (the largest value scale among its own
slots, not the cache's)."""
import numpy as np
import pytest
import torch

from oracle import kv_quant_oracle as Q
from pe_helpers import pk
from test_gpu_kv_quant import DT, Cache, attend, fresh, ints, queries

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


def check(c, layer, q, lens, K, causal=True, window=0, scale=None):
    """As the bounds of test_gpu_kv_quant.py, a row at a time: the scores' errors, 2^-11 (fp32
    queries 2^-22) a weight, fp32 sums, half a step of the output.  A weight that f16 holds in
    fewer bits, or not at all, is off by at most half of f16's smallest step, 2^-25, where the
    row's largest weight x value scale is 2^6 or more (fp32 queries 2^13): n slots lose at most
    n 2^-31 (2^-38) of 448 times the largest scale that the row sees."""
    f32 = q.dtype == torch.float32
    u = 2.0 ** -24
    out, lse = attend(c, layer, q, lens, K, causal, window, scale)
    assert c.err() == 0
    B, (_, nq, hd) = len(lens), q.shape
    q64, got, gl = (t.double().cpu().numpy() for t in (q, out, lse))
    (kc, ks), (vc, vs) = c.host("k"), c.host("v")
    kval, vval = (Q.values(x[layer, :B], y[layer, :B], c.block) for x, y in ((kc, ks), (vc, vs)))
    sc = hd ** -0.5 if scale is None else scale
    want, wl, ab = Q.attention(q64, kval, vval, lens, K, causal, window, sc)
    G = nq // kval.shape[1]
    w, tiny = (2.0 ** -22, 2.0 ** -38) if f32 else (2.0 ** -11, 2.0 ** -31)
    half = u if f32 else 2.0 ** -8
    for r in range(B * K):
        b, j = divmod(r, K)
        begin, end = Q.span(int(lens[b]), j, causal, window)
        n = end - begin
        if n <= 0:
            assert not got[r].any() and np.isneginf(gl[r]).all()
            continue
        for h in range(nq):
            g = h // G
            ak = np.abs(kval[b, g, begin:end])
            S = abs(sc) * (ak @ np.abs(q64[r, h])).max()
            d = (hd + 8) * u * S + 2.0 ** -15 + 2.0 ** -21 + 4 * u * S
            if f32:
                d += 2.0 ** -22 * S + u * abs(sc) * np.abs(q64[r, h]).max() * ak.sum(-1).max()
            top = vs[layer, b, g, begin // c.block:(end - 1) // c.block + 1].max()
            tol = ab[r, h] * (2 * d + w + 2 * (n + 64) * u) + n * tiny * 448.0 * top
            tol = tol * (1 + half) + half * np.abs(want[r, h])
            # (a tolerance of the size of the values would check nothing)
            assert tol.max() <= 2.0 ** -6 * np.abs(vval[b, g, begin:end]).max(), (r, h)
            assert (np.abs(got[r, h] - want[r, h]) <= tol).all(), (r, h)
            assert abs(gl[r, h] - wl[r, h]) <= d + (n + 64) * u + 4 * u * abs(wl[r, h]), (r, h)


def sinks(c, q, every):
    """Keys and values of a cache made anew, and queries like q: every `every`-th slot scores
    8 hd x scale above the others and has a value of zero; the others' scores are alike and their
    values positive, so what they lose adds up."""
    r = np.random.default_rng(7)
    L, B, H, cap, hd = c.shape
    u = np.where(np.arange(hd) % 3 == 0, -1.0, 1.0)
    k = r.uniform(-0.5, 0.5, c.shape)
    v = r.uniform(64.0, 448.0, c.shape)
    at = np.arange(0, cap, every)
    k[:, :, :, at], v[:, :, :, at] = 8.0 * u, 0.0
    for name, x in (("k", k), ("v", v)):
        c.t[name].copy_(torch.from_numpy(x.astype(np.float32)).cuda().to(FP8))
        c.t[name + "_scale"].fill_(1.0)
    return torch.from_numpy(u).cuda().to(q.dtype).expand(q.shape).contiguous()


# one launch, clusters, two launches, tcgen05 with heads in pieces and with more heads than SMs
@pytest.mark.parametrize("dtype,H,G,hd,K,cap,every", [
    ("bf16", 1, 8, 64, 1, 544, 32), ("f32", 1, 8, 64, 1, 544, 32), ("bf16", 3, 4, 128, 5, 2048, 32),
    ("bf16", 8, 8, 64, 8, 8192, 32), ("f32", 2, 4, 128, 4, 8192, 32),
    ("bf16", 1, 16, 64, 4, 98304, 128), ("bf16", 1, 8, 128, 5, 32768, 128)])
@pytest.mark.parametrize("nats", [13.0, 15.0, 17.0])
def test_what_a_dominated_tail_gives_is_kept(dtype, H, G, hd, K, cap, every, nats):
    """Slots that weigh e^-13 .. e^-17 of the ones beside them, alone in having values."""
    lens = [530, 100]
    c = Cache(1, 2, H, cap, hd, 32, 1, spread=0)
    q = sinks(c, torch.zeros(2 * K, H * G, hd, dtype=DT[dtype]), every)
    check(c, 0, q, lens, K, scale=nats / (8 * hd))


@pytest.mark.parametrize("hd,G,K", [(128, 1, 4), (128, 8, 5), (64, 16, 4)])
def test_a_sink_over_a_long_flat_tail(hd, G, K):
    """One slot 15 nats above 32768 others whose values are 256 times its own, a head on every SM:
    the result keeps the output's bits."""
    B, cap, nats = 160, 32768, 15.0
    g = torch.Generator("cuda").manual_seed(3)
    c = Cache.__new__(Cache)
    c.block, c.shape, c.errors = 64, (1, B, 1, cap, hd), torch.zeros(1, dtype=torch.int32, device="cuda")
    u = torch.where(torch.arange(hd, device="cuda") % 3 == 0, -1.0, 1.0)
    c.t = {"k_scale": torch.ones(1, B, 1, cap // 64, device="cuda"),
           "v_scale": torch.ones(1, B, 1, cap // 64, device="cuda")}
    for name in "kv":
        c.t[name] = torch.empty(c.shape, dtype=FP8, device="cuda")
        for b in range(B):
            x = torch.rand(cap, hd, generator=g, device="cuda")
            if name == "k":
                x = x - 0.5
                x[0] = 8.0 * u
            else:
                x = 64.0 + 384.0 * x
                x[0] = 1.0
            c.t[name][0, b, 0] = x.to(FP8)
    c.kv = pk().kv_quant_struct(c.t["k"], c.t["v"], c.t["k_scale"], c.t["v_scale"], c.errors)
    q = u.expand(B * K, G, hd).to(torch.bfloat16).contiguous()
    scale = nats / (8 * hd)
    out, lse = attend(c, 0, q, [cap - K] * B, K, scale=scale)
    assert c.err() == 0
    for b in (0, 1, 80, 151, 152, 159):
        k, v = c.t["k"][0, b, 0].double(), c.t["v"][0, b, 0].double()
        s = scale * (q.view(B, K, G, hd)[b].double() @ k.T)
        for j in range(K):
            p = s[j, :, :cap - K + j + 1].softmax(-1)
            want = p @ v[:cap - K + j + 1]
            got = out.view(B, K, G, hd)[b, j].double()
            # weights 2^-11; scores twice (hd + 12) 2^-24 x 15 + 2^-15 + 2^-21, below 2^-11; sums
            # (n + 64) 2^-23; n 2^-31 x 448 of weights that f16 holds in fewer bits; the output
            tol = want * (2.0 ** -10 + (cap + 64) * 2.0 ** -23) + cap * 2.0 ** -31 * 448.0
            tol = tol * (1 + 2.0 ** -8) + want * 2.0 ** -8
            assert ((got - want).abs() <= tol).all(), (b, j)
            ln = torch.logsumexp(s[j, :, :cap - K + j + 1], -1)
            assert ((lse.view(B, K, G)[b, j].double() - ln).abs() <= 2.0 ** -8).all()


@pytest.mark.parametrize("nq,cap,dtype", [(4, 416, "bf16"), (4, 416, "f32"), (32, 98304, "bf16")])
def test_scales_far_apart_within_what_rows_see(nq, cap, dtype):
    """Value scales over 2^+-20 in the blocks that rows see, louder ones behind them."""
    lens, K, hd, block = [400, 90], 2, 64, 16
    for seed, size in ((1, 1.0), (2, 30.0), (3, 1e-6)):
        c = Cache(1, 2, 1, cap, hd, block, seed, spread=0)
        r = np.random.default_rng(seed)
        s = 2.0 ** r.uniform(-20, 20, (1, 2, 1, cap // block))
        c.t["v_scale"].copy_(torch.from_numpy(s.astype(np.float32)))
        c.t["k_scale"].copy_(torch.from_numpy((2.0 ** r.uniform(-1, 1, s.shape)).astype(np.float32)))
        c.t["v"].view(torch.uint8)[0, :, :, 32:48] = 0
        check(c, 0, queries(2, K, nq, hd, dtype, seed, size), lens, K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("grow", [0.3, 1.0, 2.7])
def test_rows_appended_one_by_one_against_the_rows_themselves(grow, dtype):
    """Each row raises its block's scale: against the rows, not against an oracle that encodes
    again too.  2^-4 of a value for its first encoding, less than 2^-9 of the last scale for all
    others (half a step of the smallest codes, 2^-10 s, with scales that at least double)."""
    m = pk()
    B, H, hd, block, n = 2, 2, 64, 32, 32
    c = fresh(1, B, H, 64, hd, block)
    g = torch.Generator("cuda").manual_seed(2)
    size = 2.0 ** (grow * torch.arange(n, device="cuda"))
    rows = [(torch.randn(1, B, n, H, hd, device="cuda", generator=g) * size[:, None, None]).to(DT[dtype])
            for _ in "kv"]
    sl = ints([0] * B)
    for at in range(n):
        m.peagle_append_kv_quant(c.kv, B, sl, None, rows[0][:, :, at:at + 1], rows[1][:, :, at:at + 1],
                                 1, n_extra=1)
        for name, x in zip("kv", rows):
            x = x[:, :, :at + 1].double().transpose(2, 3)
            s = c.t[name + "_scale"][..., :1, None].double()
            got = c.t[name][:, :, :, :at + 1].double() * s
            assert ((got - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -9 * s).all(), (at, name)
    assert c.err() == 0 and sl.tolist() == [n] * B


# one launch, clusters, two launches, tcgen05
SCALE_SHAPES = [("bf16", 4, 416), ("f32", 4, 416), ("bf16", 4, 2048), ("f32", 8, 12288),
                ("bf16", 8, 12288), ("bf16", 32, 98304)]


@pytest.mark.parametrize("dtype,nq,cap", SCALE_SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** -80, 2.0 ** -40, 2.0 ** 120, 2.0 ** 126, 2.0 ** 127,
                                   3.4e38])
def test_value_scales_at_both_ends_of_their_range(dtype, nq, cap, scale):
    lens, K, hd = [400, 90], 2, 64
    c = Cache(1, 2, 1, cap, hd, 16, 9, spread=0)
    c.t["v"].view(torch.uint8).bitwise_and_(0xaf)  # (below 0.5: the results stay finite)
    c.t["v_scale"].fill_(scale)
    check(c, 0, queries(2, K, nq, hd, dtype, 12), lens, K)


@pytest.mark.parametrize("dtype,nq,cap", SCALE_SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126])
def test_value_scales_below_their_range_are_not_silent(dtype, nq, cap, scale):
    lens, K, hd = [400, 90], 2, 64
    c = Cache(1, 2, 1, cap, hd, 16, 9, spread=0)
    c.t["v_scale"].fill_(scale)
    out, lse = attend(c, 0, queries(2, K, nq, hd, dtype, 12), lens, K)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_whole_numbers_beyond_32_bits_are_refused():
    m = pk()
    c = Cache(1, 2, 2, 64, 64, 32, 5)
    before = {k: t.clone() for k, t in c.t.items()}
    rows = torch.zeros(2, 1, 2, 4, 2, 64, device="cuda")
    q, sl, wide = torch.zeros(2, 4, 64, device="cuda"), ints([3, 4]), 1 << 32
    out, work = torch.full_like(q, -7.0), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    saved = torch.empty(m.peagle_save_kv_quant_bytes(c.kv), dtype=torch.uint8, device="cuda")
    for call in (lambda: m.peagle_append_kv_quant(c.kv, 2, sl, None, *rows, 4, n_extra=wide + 1),
                 lambda: m.peagle_append_kv_quant(c.kv, 2, sl, None, *rows[:, 0], 4, layer=wide, n_extra=1),
                 lambda: m.peagle_append_kv_quant(c.kv, 1 - wide, sl, None, *rows, 4, n_extra=1),
                 lambda: m.peagle_append_kv_quant(c.kv, 2, sl, None, *rows, 4 - wide, n_extra=1),
                 lambda: m.peagle_read_kv_quant(c.kv, 2, sl, *rows[:, 0], 4, layer=wide),
                 lambda: m.peagle_read_kv_quant(c.kv, 2 - wide, sl, *rows, 4),
                 lambda: m.peagle_save_kv_quant(c.kv, 2, sl, saved, layer=wide),
                 lambda: m.peagle_restore_kv_quant(c.kv, 1 - wide, sl, saved),
                 lambda: m.peagle_decode_attention_quant(c.kv, wide, 2, 1, 4, q, sl, out, work),
                 lambda: m.peagle_decode_attention_quant(c.kv, 0, 2, 1, 4, q, sl, out, work, window=wide + 2)):
        with pytest.raises(m.PeagleError) as e:
            call()
        assert e.value.code == m.PEAGLE_ERR_INVALID
    torch.cuda.synchronize()
    assert sl.tolist() == [3, 4] and (out == -7.0).all() and not rows.any()
    for k, t in c.t.items():
        assert torch.equal(t.view(torch.uint8), before[k].view(torch.uint8))


def test_one_token_of_a_fused_projection_beside_a_contiguous_one():
    """Keys and values whose strides differ along axes of one element only are alike."""
    m = pk()
    B, H, hd = 1, 2, 64
    c, e = (Cache(1, B, H, 64, hd, 32, 5) for _ in "ce")
    fused = torch.randn(B, 1, 3 * H, hd, device="cuda")
    k, v = fused[:, :, :H], torch.randn(B, 1, H, hd, device="cuda")
    assert k.stride() != v.stride()
    for x, rows in ((c, (k, v)), (e, (k.contiguous(), v))):
        m.peagle_append_kv_quant(x.kv, B, ints([5]), None, *rows, 1, layer=0, n_extra=1)
    for name in c.t:
        assert torch.equal(c.t[name].view(torch.uint8), e.t[name].view(torch.uint8))
    out = torch.zeros(B, 1, 3 * H, hd, device="cuda")
    one = torch.zeros(B, 1, H, hd, device="cuda")
    m.peagle_read_kv_quant(c.kv, B, ints([1]), out[:, :, :H], one, 1, layer=0, starts=ints([5]))
    for got, x in ((out[:, :, :H], k), (one, v)):
        assert ((got - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * 8).all() and got.any()
    assert not out[:, :, H:].any() and c.err() == 0
    with pytest.raises(m.PeagleError):  # two tokens: the strides matter
        f = torch.randn(B, 2, 3 * H, hd, device="cuda")
        m.peagle_append_kv_quant(c.kv, B, ints([5]), None, f[:, :, :H], f[:, :, :H].contiguous(), 2,
                                 layer=0, n_extra=2)


def test_queries_and_output_side_by_side():
    """An output directly before and behind the queries' span is apart from it."""
    m = pk()
    B, K, nq, hd = 2, 3, 4, 64
    c = Cache(1, B, 2, 64, hd, 32, 5)
    lens = [7, 40]
    buf = torch.zeros(3, B * K, nq, hd, dtype=torch.bfloat16, device="cuda")
    buf[1] = queries(B, K, nq, hd, "bf16", 3)
    want, _ = attend(c, 0, buf[1].clone(), lens, K)
    work = torch.empty(m.peagle_decode_attention_quant_workspace(c.kv, B, K, nq), dtype=torch.uint8,
                       device="cuda")
    for i in (0, 2):
        m.peagle_decode_attention_quant(c.kv, 0, B, K, nq, buf[1], ints(lens), buf[i], work)
        assert torch.equal(buf[i], want)
    with pytest.raises(m.PeagleError):
        m.peagle_decode_attention_quant(c.kv, 0, B, K, nq, buf[1], ints(lens), buf[1], work)
    # rows so far apart that an output lies between two of them
    far = torch.zeros(B * K, 1 + B * K, nq, hd, dtype=torch.bfloat16, device="cuda")
    far[:, 0] = buf[1]
    for i in range(B * K):
        m.peagle_decode_attention_quant(c.kv, 0, B, K, nq, far[:, 0], ints(lens), far[i, 1:], work)
        assert torch.equal(far[i, 1:], want) and torch.equal(far[:, 0], buf[1])
    for out in (far.flatten(0, 1)[2:2 + B * K], far.flatten(0, 1)[B * K:2 * B * K]):
        with pytest.raises(m.PeagleError):
            m.peagle_decode_attention_quant(c.kv, 0, B, K, nq, far[:, 0], ints(lens), out, work)
