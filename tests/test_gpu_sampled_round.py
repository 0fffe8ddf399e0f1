"""Rounds of sampled speculation on the GPU, as a server makes them: the draft pass, drafts drawn from
its logits, the target's attention over the prompt that all samples share, stochastic verification, and
the commit.  Each step is held against its oracle on the inputs that it had."""
import numpy as np
import pytest
import torch

import synth
from oracle import sample_oracle as S
from oracle import shared_attn_oracle as A
from pe_helpers import make_ctx, pk, to_dev
from test_gpu_sample import DT, PROB_TOL, check_verify, dev, logits_like, of, round_of, run_sample, run_verify, settings_like,\
    struct, want_verify
from test_gpu_shared_attn import Call, bounds, check

pytestmark = pytest.mark.gpu


class Round:
    """B samples of one prompt, K drafts each.  The target is an attention over its own cache and a
    matrix; the drafter a tiny one of the library's."""

    def __init__(self, dtype, B=3, K=4, prefix=150, seed=5):
        m = pk()
        self.B, self.K, self.rows = B, K, B * (K + 1)
        self.dims = dims = synth.shrink(synth.DIMS_TINY, dtype=dtype)
        wl = synth.Workload("s", dims, B, K, (9,) * B)
        self.w = synth.make_weights(dims, seed, gains=True)
        inp = synth.make_decode_inputs(wl, seed + 1, capacity=64)
        self.ctx = make_ctx(dims, self.w, B, K, 64)
        self.d = to_dev(inp)
        self.kv = m.kv_struct(self.d["ck"], self.d["cv"], 64, B)
        vocab, dv = dims.target_vocab, dims.draft_vocab
        self.vocab, self.d2t = vocab, np.ascontiguousarray(np.asarray(self.w["d2t"]), np.int32)
        self.s = settings_like("kpm", B, seed + 2)
        self.how_draft, self.how_target = struct(self.s, K), struct(self.s, K + 1)
        self.greedy = torch.zeros(B, K, dtype=torch.int32, device="cuda")
        self.logits = torch.zeros(B, K, dv, device="cuda")
        self.tokens = torch.zeros(B * K, dtype=torch.int32, device="cuda")
        self.dist = m.sample_dist(B * K, "cuda")
        self.u = torch.zeros(B * (2 * K + 1), device="cuda")
        self.attn = Call(dtype, B, K + 1, 8, 2, 64, prefix, [20] * B, seed=seed + 3, cap=120, spare=0.5)
        g = torch.Generator("cuda").manual_seed(seed + 4)
        self.head = (torch.randn(8 * 64, vocab, generator=g, device="cuda") * 0.5).to(DT[dtype])
        self.target = torch.zeros(self.rows, vocab, device="cuda", dtype=DT[dtype])
        self.acc = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.bonus = torch.zeros_like(self.acc)
        self.commit = torch.zeros_like(self.acc)
        self.prob = torch.zeros(B, K, device="cuda")
        self.errors = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.work = torch.zeros(m.peagle_verify_sample_workspace(B, K, vocab), dtype=torch.uint8, device="cuda")

    def draw(self, seed):
        r = np.random.default_rng(seed)
        self.u.copy_(dev(r.random(self.u.numel()).astype(np.float32)))

    def run(self):
        m, B, K, c = pk(), self.B, self.K, self.attn
        n = B * K
        m.peagle_draft(self.ctx, B, self.kv, self.d["sl"], self.d["th"], self.d["nt"], K, self.greedy, self.logits)
        draft = self.logits.view(n, -1)
        m.peagle_sample(self.how_draft, draft, self.u[:n], self.tokens, d2t=dev_of(self.d2t), out_dist=self.dist,
                        errors=self.errors)
        m.peagle_decode_attention_shared(B, K + 1, c.q, c.pk, c.pv, c.plen, c.k, c.v, c.slens, c.out, c.work,
                                         out_lse=c.lse, errors=self.errors)
        torch.mm(c.out.view(self.rows, -1), self.head, out=self.target)
        m.peagle_verify_sample(B, K, self.tokens, self.how_target, self.target, self.u[n:2 * n], self.u[2 * n:],
                               self.acc, self.bonus, self.work, draft_logits=draft, draft_dist=self.dist,
                               d2t=dev_of(self.d2t), out_accept_prob=self.prob, errors=self.errors)
        torch.clamp(self.acc, max=K - 1, out=self.commit)  # (the block's rows are K)
        m.peagle_append_kv(self.ctx, B, self.kv, self.d["sl"], self.commit, n_extra=1)
        self.d["nt"].copy_(self.bonus)

    def results(self):
        return [x.clone() for x in (self.tokens, self.attn.out, self.target, self.acc, self.bonus, self.prob,
                                    self.d["sl"], self.logits)]

    def check(self):
        assert self.errors.item() == 0 and pk().peagle_status(self.ctx) == pk().PEAGLE_OK
        B, K, n, u = self.B, self.K, self.B * self.K, self.u.cpu().numpy()
        draft = self.logits.view(n, -1).cpu().numpy()
        tokens = self.tokens.cpu().numpy()
        out, lse, size = self.attn.want()
        tol, _ = bounds(self.attn, lse, size)
        assert (np.abs(self.attn.out.float().cpu().double().numpy() - out) <= tol).all()
        target = self.target.float().cpu().numpy()
        for b in range(B):
            s = of(self.s, b)
            for i in range(b * K, (b + 1) * K):
                assert tokens[i] == S.sample(draft[i], u[i], self.d2t, **s)[0]
            p = [S.distribution(x, **s) for x in target[b * (K + 1):(b + 1) * (K + 1)]]
            q = [S.spread(S.distribution(x, **s), self.d2t, self.vocab) for x in draft[b * K:(b + 1) * K]]
            m, x, a = S.verify(tokens[b * K:(b + 1) * K], p, q, u[n + b * K:n + (b + 1) * K], u[2 * n + b])
            assert (int(self.acc[b]), int(self.bonus[b])) == (m, x)
            assert (np.abs(self.prob[b].cpu().double().numpy() - a) <= 2 * PROB_TOL * a).all()


TABLES = {}


def dev_of(a):
    """One device copy of a table: a graph reads it again when it is replayed."""
    key = a.tobytes()
    if key not in TABLES:
        TABLES[key] = dev(a)
    return TABLES[key]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rounds(dtype):
    r = Round(dtype)
    lens = r.d["sl"].cpu().numpy()
    for step in range(4):
        r.draw(step)
        r.run()
        r.check()
        now = r.d["sl"].cpu().numpy()
        assert np.array_equal(now, lens + 1 + np.minimum(r.acc.cpu().numpy(), r.K - 1))
        lens = now
        # the target's own cache grows as well
        r.attn.lens = [int(x) for x in np.asarray(r.attn.lens) + 1 + r.acc.cpu().numpy()]
        r.attn.slens.copy_(torch.tensor(r.attn.lens, dtype=torch.int32))
    r.ctx.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_captured_round_is_the_eager_round(dtype):
    r = Round(dtype, seed=6)
    first = [x.clone() for x in (r.d["ck"], r.d["cv"], r.d["sl"], r.d["nt"])]

    def again():
        for x, y in zip((r.d["ck"], r.d["cv"], r.d["sl"], r.d["nt"]), first):
            x.copy_(y)

    want = []
    for step in range(3):
        r.draw(10 + step)
        r.run()
        want.append(r.results())
    again()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.run()
    again()
    for step in range(3):
        r.draw(10 + step)
        r.acc.fill_(-5)
        r.tokens.fill_(-5)
        g.replay()
        for x, y in zip(r.results(), want[step]):
            assert torch.equal(x, y)
    r.check()
    r.ctx.close()


def test_two_verifications_at_once():
    """Two streams, a workspace each; and each stream's own sampling before it."""
    a, b = round_of(5, 4, 30011, 9001, "bf16", "kpm", 41), round_of(40, 8, 5003, 5003, "f32", "p", 42)
    want = [run_verify(t) for t in (a, b)]
    m, outs, streams = pk(), [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for t in (a, b):
        n, B, K = t["B"] * t["K"], t["B"], t["K"]
        i32 = dict(dtype=torch.int32, device="cuda")
        outs.append(dict(tokens=torch.zeros(n, **i32), dist=m.sample_dist(n, "cuda"), acc=torch.zeros(B, **i32),
                         bonus=torch.zeros(B, **i32), prob=torch.zeros(B, K, device="cuda"), d2t=dev(t["d2t"]),
                         u=[dev(t[k]) for k in ("u_draft", "u_accept", "u_bonus")],
                         how=[struct(t["s"], K), struct(t["s"], K + 1)],
                         work=torch.zeros(m.peagle_verify_sample_workspace(B, K, t["vocab"]), dtype=torch.uint8,
                                          device="cuda")))
    torch.cuda.synchronize()
    for _ in range(10):
        for t, o, s in zip((a, b), outs, streams):
            m.peagle_sample(o["how"][0], t["draft"], o["u"][0], o["tokens"], d2t=o["d2t"], out_dist=o["dist"], stream=s)
            m.peagle_verify_sample(t["B"], t["K"], o["tokens"], o["how"][1], t["target"], o["u"][1], o["u"][2],
                                   o["acc"], o["bonus"], o["work"], draft_logits=t["draft"], draft_dist=o["dist"],
                                   d2t=o["d2t"], out_accept_prob=o["prob"], stream=s)
    torch.cuda.synchronize()
    for t, o, w in zip((a, b), outs, want):
        assert np.array_equal(o["tokens"].cpu().numpy(), t["tokens"])
        assert np.array_equal(o["acc"].cpu().numpy(), w[0]) and np.array_equal(o["bonus"].cpu().numpy(), w[1])
        assert np.array_equal(o["prob"].cpu().double().numpy(), w[2])


@pytest.mark.parametrize("which", ["", "kp"])
def test_verify_more_rows_than_are_listed(which):
    """Above 16384 rows no lists are kept."""
    t = round_of(520, 32, 97, 61, "f32", which, 43, permute=True)
    assert t["B"] * (t["K"] + 1) > 16384
    acc, bonus, prob = run_verify(t)
    for b in range(0, t["B"], 13):
        m, x, a = want_verify(t, b)
        assert (acc[b], bonus[b]) == (m, x)
        assert (np.abs(prob[b] - a) <= 2 * PROB_TOL * a).all()


def test_verify_long_and_short_rows_side_by_side():
    """top-k in the same batch off, longer than a list, and short; many rows at once."""
    t = round_of(30, 5, 40009, 32000, "bf16", "kp", 44, noise=0.2)
    t["s"]["top_k"] = np.resize(np.array([0, 20, 600, 448, 1], np.int32), 30)
    t["tokens"], _, t["dist"] = run_sample(t["draft"], t["u_draft"], t["s"], t["d2t"], 5)
    check_verify(t)


# ------------------------------------------------------------------ attention: references that jump

JUMPS = {"rising": [0, 4, 30, 60], "falling": [60, 30, 4, 0], "far": [0, 50, 0, 110], "low first": [-90, 0, 0, 0],
         "steps": [0, 20, 41, 20, 62, 82, 60, 103], "up and down": [0, 12, -40, 12, 24, -100, 36, 70, 0]}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("jumps", sorted(set(JUMPS) - {"steps"}))
@pytest.mark.parametrize("prefix,lens", [(1100, [3, 200]), (0, [700, 1000, 0])])
def test_scores_that_jump_between_tiles(prefix, lens, jumps, hd, dtype):
    """Every row's scores step by up to 110 (2^159) from one stretch of 128 slots to the next."""
    check(jumping(dtype, hd, prefix, lens, jumps))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
def test_large_values_while_scores_jump(hd, dtype):
    """Weights up to 2^32 meet values of 2^68 and some more before the reference follows."""
    c = jumping(dtype, hd, 1100, [3, 200], "steps")
    for t in (c.pv, c.v):
        t.mul_(2.0 ** 68)
    check(c)


def jumping(dtype, hd, prefix, lens, jumps):
    c = Call(dtype, len(lens), 4, 8, 2, hd, prefix, lens)
    way = torch.zeros(hd, device="cuda", dtype=c.q.dtype)
    way[::2] = 1.0
    c.q.mul_(0.25).add_(way)  # (scores of the step alone: jump x 0.5 hd / sqrt(hd))
    steps = JUMPS[jumps]
    unit = 1 / (0.5 * hd ** 0.5)
    for t in (c.pk[:, :prefix], *[c.k[b:b + 1, :, :max(n + 4, 1)] for b, n in enumerate(lens)]):
        n = t.shape[-2]
        if n:
            add = torch.tensor([steps[i // 128 % len(steps)] for i in range(n)], device="cuda") * unit
            t += (add[:, None] * way.float()).to(t.dtype)
    return c
