"""Sampling and the verification of sampled drafts on the GPU against their fp64 oracle.  Tokens and
counts are equal.  A probability is w / S in fp32: it is off by its rounding (2^-24 of it) and by
the sum of the kept weights, whole numbers of 2^-F of the largest: vocab x 2^-(F+1) <= 2^-27 of S,
which is at least the largest, and 2^-36 for the weights themselves."""
import numpy as np
import pytest
import torch

import synth
from oracle import sample_oracle as S
from pe_helpers import make_ctx, pk, run_draft

pytestmark = pytest.mark.gpu
PROB_TOL = 2.0 ** -24 + 2.0 ** -26  # relative
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def logits_like(kind, rows, vocab, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, vocab)) * 2.2
    if kind == "model":
        for row in x:
            at = r.integers(0, vocab, 24)
            row[at] += 5 + 3 * r.exponential(size=24)
    elif kind == "ties":  # few values: every border falls among equal logits
        x = np.round(x)
    elif kind == "same":
        x[:] = r.standard_normal((rows, 1))
    elif kind == "zeros":  # -0 and +0 are equal
        x = np.where(r.random((rows, vocab)) < 0.5, -0.0, 0.0)
    elif kind == "masked":
        x[r.random((rows, vocab)) < 0.9] = -np.inf
        x[np.arange(rows), r.integers(0, vocab, rows)] = 1.0
    elif kind == "alone":
        x[:] = -np.inf
        x[np.arange(rows), r.integers(0, vocab, rows)] = -3.0
    elif kind == "huge":
        x *= 1e37
    elif kind == "tiny":
        x *= 1e-40
    elif kind == "far":  # a large common part: differences of a few last places
        x = 4096.0 + np.round(x * 64) / 512
    return x.astype(np.float32)


def settings_like(which, n, seed):
    r = np.random.default_rng(seed)
    s = {"temperature": r.choice([0.25, 0.7, 1.0, 1.7], n).astype(np.float32)}
    if "k" in which:
        s["top_k"] = r.choice([1, 2, 7, 50, 300, 1000], n).astype(np.int32)
    if "p" in which:
        s["top_p"] = r.choice([0.05, 0.5, 0.9, 0.999], n).astype(np.float32)
    if "m" in which:
        s["min_p"] = r.choice([0.001, 0.05, 0.4, 1.0], n).astype(np.float32)
    return s


def struct(s, rows_per=1):
    return pk().sampling_struct(**{k: dev(v) for k, v in s.items()}, rows_per=rows_per)


def of(s, r):
    return {k: v[r] for k, v in s.items()}


def run_sample(x, u, s, d2t=None, rows_per=1, dist=True, errors=None):
    """x a CUDA tensor [rows, vocab]; returns tokens, probabilities and the records."""
    n = x.shape[0]
    token = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((n,), -7.0, device="cuda")
    d = pk().sample_dist(n, "cuda") if dist else None
    pk().peagle_sample(None if s is None else struct(s, rows_per), x, dev(u), token, out_prob=prob,
                       d2t=None if d2t is None else dev(d2t), out_dist=d, errors=errors)
    return token.cpu().numpy(), prob.cpu().double().numpy(), d


def check_sample(x, u, s, d2t=None, rows_per=1):
    token, prob, dist = run_sample(x, u, s, d2t, rows_per)
    host = x.float().cpu().numpy()
    index = dist.view(torch.int32)[:, 6].cpu().numpy()
    for r in range(len(host)):
        t, p, i = S.sample(host[r], u[r], d2t, **({} if s is None else of(s, r // rows_per)))
        assert (token[r], index[r]) == (t, i), (r, None if s is None else of(s, r // rows_per))
        assert abs(prob[r] - p) <= PROB_TOL * p, r


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 500, 4097, 32000])
@pytest.mark.parametrize("which", ["", "k", "p", "m", "kpm"])
def test_sample(vocab, which, dtype):
    rows = 9
    x = dev(logits_like("model", rows, vocab, vocab), DT[dtype])
    u = np.random.default_rng(1).random(rows).astype(np.float32)
    check_sample(x, u, settings_like(which, rows, 2 + vocab))


@pytest.mark.parametrize("kind", ["ties", "same", "zeros", "masked", "alone", "huge", "tiny", "far"])
@pytest.mark.parametrize("which", ["", "k", "p", "kpm"])
@pytest.mark.parametrize("rows,vocab", [(6, 1000), (3, 40001)])
def test_sample_where_borders_fall_badly(rows, vocab, which, kind):
    x = dev(logits_like(kind, rows, vocab, 5))
    u = np.random.default_rng(6).random(rows).astype(np.float32)
    check_sample(x, u, settings_like(which, rows, 7))


@pytest.mark.parametrize("vocab,dtype", [(201088, "f32"), (201088, "bf16"), (262144, "f32"), (262143, "bf16")])
@pytest.mark.parametrize("kind", ["model", "bulk", "ties"])
def test_sample_large_vocabularies(kind, vocab, dtype):
    rows = 5
    x = dev(logits_like(kind, rows, vocab, 8), DT[dtype])
    u = np.random.default_rng(9).random(rows).astype(np.float32)
    for which in ("", "kp", "pm"):
        check_sample(x, u, settings_like(which, rows, 10))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_at_any_stride_and_alignment(dtype):
    """Rows of a wider buffer, starting at odd elements; what lies between them is not read as part
    of a row, and the bits do not depend on where a row lies or how many rows there are."""
    rows, vocab = 7, 1531
    base = logits_like("model", rows, vocab, 11)
    u = np.random.default_rng(12).random(rows).astype(np.float32)
    s = settings_like("kpm", rows, 13)
    x = dev(base, DT[dtype])
    want = run_sample(x, u, s)
    for stride, at in ((1531, 1), (1540, 3), (2000, 0), (1533, 5)):
        wide = torch.full((rows * stride + 8,), float("nan"), device="cuda", dtype=DT[dtype])
        view = wide[at:at + rows * stride].view(rows, stride)[:, :vocab]
        view.copy_(x)
        got = run_sample(view, u, s)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert torch.equal(got[2], want[2])
    for r in (0, 6):
        got = run_sample(x[r:r + 1], u[r:r + 1], {k: v[r:r + 1] for k, v in s.items()})
        assert got[0][0] == want[0][r] and torch.equal(got[2][0], want[2][r])


def test_random_numbers_at_their_ends():
    vocab = 6000
    x = logits_like("model", 1, vocab, 14)
    x[0, :3] = -np.inf
    x[0, -2:] = -np.inf
    u = np.array([0.0, -1.0, np.nan, 1 - 2.0 ** -24, 1.0, 7.0, np.inf], np.float32)
    token, prob, _ = run_sample(dev(np.repeat(x, len(u), 0)), u, None)
    p = S.distribution(x[0])
    live = np.nonzero(p > 2.0 ** -44)[0]
    assert (token[:3] == live[0]).all()
    assert (token[4:] == live[-1]).all() and token[3] == S.pick(p, u[3])


def test_greedy_rows_and_rows_without_a_distribution():
    vocab = 5000
    x = logits_like("ties", 9, vocab, 15)
    x[1, 17] = np.nan
    x[2, 4999] = -np.nan
    x[3, 0] = np.inf
    x[4] = -np.inf
    T = np.array([0.0, 1, 1, 1, 1, -1.0, np.nan, 1e-30, np.inf], np.float32)
    u = np.full(9, 0.3, np.float32)
    errors = torch.zeros(1, dtype=torch.int32, device="cuda")
    token, prob, dist = run_sample(dev(x), u, {"temperature": T}, errors=errors)
    assert token[0] == np.argmax(x[0]) and prob[0] == 1 and token[7] == np.argmax(x[7])
    assert (token[1:7] == -1).all() and np.isnan(prob[1:7]).all()
    assert (dist[1:7, :8] == 0).all() and errors.item() == pk().PEAGLE_DEV_BAD_ROW
    assert token[8] == int(np.float32(0.3) * np.float64(vocab)) and abs(prob[8] - 1 / vocab) < 1e-9
    errors.zero_()
    run_sample(dev(x[7:]), u[7:], {"temperature": T[7:]}, errors=errors)
    assert errors.item() == 0


@pytest.mark.parametrize("rows,vocab", [(1, 33), (300, 700), (40, 4096)])
def test_settings_out_of_range_are_off_or_clamped(rows, vocab):
    x = dev(logits_like("model", rows, vocab, 16))
    u = np.random.default_rng(17).random(rows).astype(np.float32)
    r = np.random.default_rng(18)
    s = {"temperature": np.ones(rows, np.float32),
         "top_k": r.choice([-5, 0, vocab, vocab + 1, 2 ** 31 - 1, 3], rows).astype(np.int32),
         "top_p": r.choice([-1.0, 0.0, 1.0, 2.0, np.nan, np.inf, 0.8], rows).astype(np.float32),
         "min_p": r.choice([-1.0, 0.0, np.nan, 2.0, 0.1], rows).astype(np.float32)}
    check_sample(x, u, s)


def test_rows_share_settings_and_map_through_d2t():
    B, K, vocab = 5, 7, 900
    x = dev(logits_like("model", B * K, vocab, 19))
    u = np.random.default_rng(20).random(B * K).astype(np.float32)
    d2t = (np.sort(np.random.default_rng(21).permutation(5000)[:vocab]) - np.arange(vocab)).astype(np.int32)
    check_sample(x, u, settings_like("kpm", B, 22), d2t, rows_per=K)


# ---------------------------------------------------------------- verification

def round_of(B, K, vocab, dv, dtype, which, seed, greedy=False, permute=False, kind="model", noise=0.7):
    """One round: target and draft logits, drafts drawn by peagle_sample (or greedy ones)."""
    r = np.random.default_rng(seed)
    target = logits_like(kind, B * (K + 1), vocab, seed)
    ids = r.permutation(vocab)[:dv] if permute else np.sort(r.permutation(vocab)[:dv])
    d2t = (ids - np.arange(dv)).astype(np.int32)
    draft = target.reshape(B, K + 1, vocab)[:, :K].reshape(B * K, vocab)[:, ids]
    with np.errstate(invalid="ignore"):
        draft = (draft + noise * r.standard_normal(draft.shape)).astype(np.float32)
    s = settings_like(which, B, seed + 1)
    t = {"target": dev(target, DT[dtype]), "draft": dev(draft), "d2t": d2t, "s": s, "K": K, "B": B,
         "u_draft": r.random(B * K).astype(np.float32), "u_accept": r.random(B * K).astype(np.float32),
         "u_bonus": r.random(B).astype(np.float32), "vocab": vocab, "greedy": greedy}
    ds = {"temperature": np.zeros(B, np.float32)} if greedy else s
    t["tokens"], _, t["dist"] = run_sample(t["draft"], t["u_draft"], ds, d2t, K)
    return t


def run_verify(t, errors=None, stream=None, work=None):
    m, B, K = pk(), t["B"], t["K"]
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    bonus, prob = torch.full_like(acc, -7), torch.full((B, K), -7.0, device="cuda")
    if work is None:
        work = torch.full((m.peagle_verify_sample_workspace(B, K, t["vocab"]),), 0xff, dtype=torch.uint8,
                          device="cuda")
    g = t["greedy"]
    m.peagle_verify_sample(B, K, dev(t["tokens"].astype(np.int32)), struct(t["s"], K + 1), t["target"],
                           dev(t["u_accept"]), dev(t["u_bonus"]), acc, bonus, work,
                           draft_logits=None if g else t["draft"], draft_dist=None if g else t["dist"],
                           d2t=None if g else dev(t["d2t"]), out_accept_prob=prob, errors=errors)
    return acc.cpu().numpy(), bonus.cpu().numpy(), prob.cpu().double().numpy()


def want_verify(t, b):
    K, vocab = t["K"], t["vocab"]
    x = t["target"][b * (K + 1):(b + 1) * (K + 1)].float().cpu().numpy()
    p = [S.distribution(row, **of(t["s"], b)) for row in x]
    tokens = t["tokens"][b * K:(b + 1) * K]
    if t["greedy"]:
        q = [np.eye(1, vocab, max(int(i), 0))[0] for i in tokens]
    else:
        d = t["draft"][b * K:(b + 1) * K].cpu().numpy()
        q = [S.spread(S.distribution(row, **of(t["s"], b)), t["d2t"], vocab) for row in d]
    return S.verify(tokens, p, q, t["u_accept"][b * K:(b + 1) * K], t["u_bonus"][b])


def check_verify(t):
    acc, bonus, prob = run_verify(t)
    for b in range(t["B"]):
        m, x, a = want_verify(t, b)
        assert (acc[b], bonus[b]) == (m, x), (b, of(t["s"], b))
        assert (np.abs(prob[b] - a) <= 2 * PROB_TOL * a).all(), b  # two such probabilities
    return acc


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,K,vocab,dv", [(1, 1, 2, 1), (3, 4, 37, 37), (5, 8, 5001, 1500), (2, 16, 32000, 32000),
                                          (4, 33, 700, 300), (2, 64, 300, 40)])
@pytest.mark.parametrize("which", ["", "kpm"])
def test_verify(B, K, vocab, dv, which, dtype):
    check_verify(round_of(B, K, vocab, dv, dtype, which, 23, noise=0.3))


@pytest.mark.parametrize("permute", [False, True])
def test_verify_a_large_vocabulary(permute):
    t = round_of(3, 8, 201088, 32000, "bf16", "p", 24, permute=permute, noise=0.2)
    check_verify(t)


def test_verify_greedy_drafts():
    t = round_of(6, 5, 3001, 2000, "f32", "k", 25, greedy=True)
    check_verify(t)


@pytest.mark.parametrize("kind", ["ties", "same", "masked", "alone", "far"])
def test_verify_where_borders_fall_badly(kind):
    check_verify(round_of(5, 4, 2003, 1000, "f32", "kp", 26, kind=kind, permute=True))
    check_verify(round_of(5, 4, 2003, 2003, "f32", "", 27, kind=kind))


def test_a_drafter_that_is_the_target_is_always_accepted():
    t = round_of(4, 6, 4000, 4000, "f32", "kpm", 28, noise=0.0)
    t["u_accept"][:] = 1 - 2.0 ** -24
    acc, _, prob = run_verify(t)
    assert (acc == 6).all() and (prob == 1).all()


def test_verify_at_temperature_zero_is_verify_greedy():
    t = round_of(6, 5, 3000, 3000, "f32", "", 29, noise=0.2)
    t["s"] = {"temperature": np.zeros(6, np.float32)}
    t["tokens"], _, t["dist"] = run_sample(t["draft"], t["u_draft"], t["s"], t["d2t"], 5)
    acc, bonus, _ = run_verify(t)
    got = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    best = t["target"].argmax(-1).int().view(6, 6)
    pk().peagle_verify_greedy(6, 5, dev(t["tokens"].astype(np.int32)), best, *got)
    assert np.array_equal(acc, got[0].cpu().numpy()) and np.array_equal(bonus, got[1].cpu().numpy())


def test_first_token_has_the_targets_distribution():
    """4096 requests that differ only in their random numbers: the first token that comes out is
    distributed as the target's, whatever the drafter's distribution.  Five standard deviations of a
    multinomial count each, for 12 tokens."""
    B, vocab = 4096, 12
    r = np.random.default_rng(30)
    t = {"B": B, "K": 1, "vocab": vocab, "greedy": False, "d2t": np.zeros(vocab, np.int32),
         "s": {"temperature": np.full(B, 0.9, np.float32)}}
    one, other = r.standard_normal((2, 1, vocab)).astype(np.float32) * 1.5
    t["target"] = dev(np.repeat(one, 2 * B, 0))
    t["draft"] = dev(np.repeat(other, B, 0))
    for name, n in (("u_draft", B), ("u_accept", B), ("u_bonus", B)):
        t[name] = r.random(n).astype(np.float32)
    t["tokens"], _, t["dist"] = run_sample(t["draft"], t["u_draft"], t["s"], t["d2t"])
    acc, bonus, _ = run_verify(t)
    first = np.where(acc > 0, t["tokens"], bonus)
    p = S.distribution(one[0], 0.9)
    n = np.bincount(first, minlength=vocab)
    assert (np.abs(n - B * p) <= 5 * np.sqrt(B * p * (1 - p)) + 1).all()
    assert 0.2 < acc.mean() < 0.95


def test_bad_tokens_records_and_rows_are_rejected():
    m, K = pk(), 4
    t = round_of(7, K, 900, 900, "f32", "", 31, noise=0.0)
    t["u_accept"][:] = 0.0
    tokens = t["tokens"].reshape(7, K)
    tokens[0, 2] = 900
    tokens[1, 0] = -1
    tokens[2, 3] = (tokens[2, 3] + 1) % 900  # not its record's
    rows = t["target"].view(7, K + 1, 900)
    rows[3, 1] = float("nan")
    rows[4, 4, 5] = float("inf")
    t["tokens"] = tokens.reshape(-1)
    d = t["draft"].view(7, K, 900)
    d[5, 2, 0] = float("nan")
    keep, t["tokens"] = t["tokens"], None
    token, _, t["dist"] = run_sample(t["draft"], t["u_draft"], t["s"], t["d2t"], K)
    t["tokens"] = keep
    errors = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, bonus, prob = run_verify(t, errors)
    assert acc.tolist() == [2, 0, 3, 1, 4, 2, 4]
    assert bonus[3] == -1 and bonus[4] == -1 and (bonus[[0, 1, 2, 5, 6]] >= 0).all()
    assert prob[0, 2] == prob[1, 0] == prob[2, 3] == prob[3, 1] == prob[5, 2] == 0
    assert errors.item() == m.PEAGLE_DEV_BAD_TOKEN | m.PEAGLE_DEV_BAD_ROW
    for b in (0, 1, 2, 5):  # drawn from p itself
        x = rows[b, acc[b]].cpu().numpy()
        assert bonus[b] == S.pick(S.distribution(x, **of(t["s"], b)), t["u_bonus"][b])
