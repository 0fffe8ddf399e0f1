"""Sampling from many rows at once, where a CTA passes by a row once and a cluster takes what that leaves,
against the 64-bit oracle, as few rows are."""
import numpy as np
import pytest
import torch

from test_gpu_sample import DT, check_sample, dev, logits_like, run_sample, settings_like

pytestmark = pytest.mark.gpu

ROWS = 203


def rising(rows, vocab, seed):
    """Logits that rise along the row, so that no token seen early stays among the first k."""
    r = np.random.default_rng(seed)
    return (np.linspace(-9, 9, vocab)[None] + 0.01 * r.standard_normal((rows, vocab))).astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [4097, 9001, 40003])
@pytest.mark.parametrize("which", ["k", "kp", "kpm"])
def test_many_rows(vocab, which, dtype):
    x = dev(logits_like("model", ROWS, vocab, vocab), DT[dtype])
    u = np.random.default_rng(1).random(ROWS).astype(np.float32)
    check_sample(x, u, settings_like(which, ROWS, 2 + vocab))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["same", "ties", "zeros", "masked", "alone", "far", "huge", "rising"])
def test_many_rows_where_borders_fall_badly(kind, dtype):
    vocab = 36871
    x = rising(ROWS, vocab, 3) if kind == "rising" else logits_like(kind, ROWS, vocab, 3)
    u = np.random.default_rng(4).random(ROWS).astype(np.float32)
    s = settings_like("kpm", ROWS, 5)
    s["top_k"] = np.resize(np.array([1, 2, 40, 300, 448, 449, 512, 513, 2000, vocab - 1], np.int32), ROWS)
    check_sample(dev(x, DT[dtype]), u, s)


@pytest.mark.parametrize("rows", [1, 9, ROWS])
@pytest.mark.parametrize("lead", [40.0, 1e4, 1e30])
def test_tokens_far_above_the_others(rows, lead):
    """A few tokens lead by far: top-k still keeps the first of those that have no weight beside them."""
    vocab = 33001
    x = logits_like("model", rows, vocab, 20)
    x[:, 100:103] = lead * np.array([1.0, 0.999, 1.0], np.float32)
    u = np.random.default_rng(21).random(rows).astype(np.float32)
    s = settings_like("kp", rows, 22)
    s["temperature"] = np.resize(np.array([0.05, 0.7, lead / 10], np.float32), rows)
    check_sample(dev(x), u, s)


@pytest.mark.parametrize("rows", [1, 9, ROWS])
@pytest.mark.parametrize("top_k", [2, 300])
def test_fewer_tokens_than_top_k(rows, top_k):
    """All but one, or three equal ones, of the tokens are masked."""
    vocab = 33001
    x = np.full((rows, vocab), -np.inf, np.float32)
    x[:, 5] = -2.5
    x[::2, 16000] = x[::2, 32999] = -2.5
    x[::3, 16001] = -3.5
    u = np.random.default_rng(23).random(rows).astype(np.float32)
    check_sample(dev(x), u, {"top_k": np.full(rows, top_k, np.int32)})


@pytest.mark.parametrize("rows,vocab,dtype", [(77, 201088, "bf16"), (41, 262144, "f32")])
def test_many_rows_of_large_vocabularies(rows, vocab, dtype):
    """Clusters of 4 and 8 with rows of both kinds, and places behind the last row."""
    x = dev(logits_like("model", rows, vocab, 17), DT[dtype])
    u = np.random.default_rng(18).random(rows).astype(np.float32)
    s = settings_like("kpm", rows, 19)
    s["top_k"] = np.resize(np.array([0, 20, 1000, 50, 1, 448, 60000, 3, vocab], np.int32), rows)
    check_sample(x, u, s)


@pytest.mark.parametrize("top_k", [0, 1, 50, 448, 449, 5000])
def test_many_rows_with_one_top_k(top_k):
    """What top-k leaves (nothing cut, one token, more than a list holds), with top-p and without."""
    vocab = 20011
    x = dev(logits_like("model", ROWS, vocab, 6))
    u = np.random.default_rng(7).random(ROWS).astype(np.float32)
    r = np.random.default_rng(8)
    check_sample(x, u, {"top_k": np.full(ROWS, top_k, np.int32),
                        "top_p": r.choice([1.0, 0.9, 0.5], ROWS).astype(np.float32),
                        "temperature": r.choice([0.0, 0.3, 1.0, 1.7], ROWS).astype(np.float32)})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_at_any_alignment(dtype):
    vocab = 6007
    base = logits_like("model", ROWS, vocab, 9)
    u = np.random.default_rng(10).random(ROWS).astype(np.float32)
    s = settings_like("kp", ROWS, 11)
    first = None
    for stride, at in [(vocab, 0), (vocab + 1, 1), (vocab + 5, 3)]:
        wide = torch.full((ROWS * stride + 8,), float("nan"), device="cuda", dtype=DT[dtype])
        view = wide[at:at + ROWS * stride].view(ROWS, stride)[:, :vocab]
        view.copy_(dev(base))
        got = run_sample(view, u, s)[:2]
        if first is None:
            first = got
            check_sample(view, u, s)
        assert np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1])


def test_many_rows_equal_few_rows():
    """A row's result does not depend on how many rows there are."""
    vocab = 50021
    x = dev(logits_like("model", ROWS, vocab, 12), torch.bfloat16)
    u = np.random.default_rng(13).random(ROWS).astype(np.float32)
    s = settings_like("kpm", ROWS, 14)
    token, prob, dist = run_sample(x, u, s)
    for lo in range(0, ROWS, 29):
        part = {k: v[lo:lo + 29] for k, v in s.items()}
        t, p, d = run_sample(x[lo:lo + 29], u[lo:lo + 29], part)
        assert np.array_equal(t, token[lo:lo + 29]) and np.array_equal(p, prob[lo:lo + 29])


def test_many_rows_without_a_distribution():
    vocab = 8193
    x = logits_like("model", ROWS, vocab, 15)
    bad = {3: np.nan, 50: np.inf, 77: -np.inf, 202: np.nan}
    for r, v in bad.items():
        if v == -np.inf:
            x[r] = v
        else:
            x[r, (r * 97) % vocab] = v
    errors = torch.zeros(1, dtype=torch.int32, device="cuda")
    u = np.full(ROWS, 0.5, np.float32)
    s = settings_like("k", ROWS, 16)
    s["top_k"][:] = 20
    token, prob, _ = run_sample(dev(x), u, s, errors=errors)
    assert int(errors.item()) != 0
    for r in range(ROWS):
        assert (token[r] == -1) == (r in bad) and np.isnan(prob[r]) == (r in bad)
