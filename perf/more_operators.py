"""Sampled speculative rounds: what their operators compute, on which sizes they are measured.

A round at a temperature draws the drafts from the drafter's logits, verifies them so that what
comes out is distributed as the target's own samples, and, where several samples of one prompt
run side by side, attends over the prompt's keys and values that they share.

  sample     a row of logits -> temperature, top-k, top-p and min-p -> the token that a given
             random number picks, and its probability
  verify     K drafts a request against the target's distributions: the accepted prefix, the
             token after it (from what the drafter left of the target's distribution), and the
             probability with which each draft is accepted
  attention  K draft rows a request over one prefix that the batch shares and over the
             request's own slots behind it, for one layer

``run`` computes them in elementary torch operations, or, where ``own`` is set, through the
package's entry points.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases

def _sample(name, dtype, rows, vocab, per, temperature, top_k=0, top_p=1.0, min_p=0.0, target=0, flat=0.0):
    return {"name": name, "op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab, "per": per,
            "temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p, "target": target,
            "flat": flat}


def _verify(name, dtype, batch, K, vocab, draft_vocab, temperature, top_k=0, top_p=1.0, min_p=0.0, greedy=False):
    return {"name": name, "op": "verify", "dtype": dtype, "batch": batch, "K": K, "vocab": vocab,
            "draft_vocab": draft_vocab, "temperature": temperature, "top_k": top_k, "top_p": top_p,
            "min_p": min_p, "greedy": greedy}


def _attn(name, dtype, heads, kv_heads, head_dim, batch, K, prefix, lo, hi, causal=True):
    return {"name": name, "op": "attention", "dtype": dtype, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "batch": batch, "K": K, "prefix": prefix, "lo": lo, "hi": hi,
            "causal": causal}


def listed():
    return [
        # the tiny drafter's four draft rows: latency alone
        _sample("sample_tiny", "f32", 4, 4096, 4, 0.8, top_k=50),
        # a draft pass of one request over the pruned vocabulary, mapped into the target's
        _sample("sample_draft_b1", "f32", 8, 32000, 8, 1.0, top_p=0.95, target=201088),
        # the drafts of 64 requests
        _sample("sample_draft_b64", "f32", 512, 32000, 8, 0.7, top_k=200, top_p=0.9, min_p=0.02, target=201088),
        # one token of the target for each of 64 requests, as its head leaves the logits
        _sample("sample_target_b64", "bf16", 64, 201088, 1, 0.9, top_k=64, top_p=0.95),
        # a hot, nearly flat distribution: thousands of tokens stay in
        _sample("sample_hot_b16", "f32", 16, 201088, 1, 1.6, top_p=0.99, flat=0.7),
        # one request verified
        _verify("verify_b1", "f32", 1, 8, 201088, 32000, 0.8, top_p=0.95),
        # 16 requests of the wide drafter, one vocabulary for both models
        _verify("verify_b16", "f32", 16, 5, 32000, 32000, 1.0),
        # 64 requests, target logits in 16 bits, filters that keep few tokens
        _verify("verify_b64", "bf16", 64, 8, 201088, 32000, 0.7, top_k=100, top_p=0.9),
        # two samples of a short prompt, the tiny fp32 drafter
        _attn("attn_tiny", "f32", 4, 2, 64, 2, 4, 128, 5, 16),
        # four samples of a prompt of 4096 tokens, the H=2880 drafter
        _attn("attn_b4", "bf16", 64, 8, 64, 4, 8, 4096, 17, 301),
        # 64 samples of a long prompt
        _attn("attn_b64", "bf16", 64, 8, 64, 64, 8, 8192, 1, 1023),
        # one token each for 16 readers of a long document, the wide drafter's heads
        _attn("attn_long_token", "bf16", 32, 8, 128, 16, 1, 131071, 33, 2049),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _filters(rng, vocab):
    return {"temperature": rng.choice([0.3, 0.7, 1.0, 1.0, 1.3, rng.uniform(0.2, 2.0)]),
            "top_k": rng.choice([0, 0, _log(rng, 1, min(vocab, 2000))]),
            "top_p": rng.choice([1.0, 0.9, 0.95, rng.uniform(0.1, 0.999)]),
            "min_p": rng.choice([0.0, 0.0, 0.05, rng.uniform(0.001, 0.5)])}


def draw(rng):
    op = rng.choice(["sample", "verify", "attention"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "sample":
        vocab = _log(rng, 500, 262144)
        rows = _log(rng, 1, max(2, min(512, 12000000 // vocab)))
        c = {"op": op, "dtype": dtype, "rows": rows, "vocab": vocab, "per": rng.choice([1, 1, 5, 8]),
             "target": rng.choice([0, vocab + rng.randint(1, 3 * vocab)]),
             "flat": rng.choice([0.0, 0.0, rng.uniform(0.1, 0.9)])}
        return {**c, **_filters(rng, vocab)}
    if op == "verify":
        vocab = _log(rng, 500, 262144)
        K = rng.randint(1, 16)
        batch = _log(rng, 1, max(2, min(64, 100000000 // (vocab * (K + 1)))))
        c = {"op": op, "dtype": dtype, "batch": batch, "K": K, "vocab": vocab,
             "draft_vocab": rng.choice([vocab, rng.randint(vocab // 8, vocab)]),
             "greedy": rng.random() < 0.25}
        return {**c, **_filters(rng, vocab)}
    head_dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    K = rng.randint(1, min(16, 128 // group))
    batch = _log(rng, 1, 64)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    # products at most about those of the largest listed case (16th of it in 32 bits)
    products = int(7e10) if dtype == "bf16" else int(4e9)
    most = products // (4 * head_dim * kv_heads * group * batch * K)
    prefix = _log(rng, 1, max(2, min(131072, most)))
    hi = _log(rng, 1, max(2, min(4096, most, 2 ** 28 // (batch * kv_heads * head_dim))))
    return {"op": op, "dtype": dtype, "heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim,
            "batch": batch, "K": K, "prefix": prefix, "lo": max(1, int(hi * rng.uniform(0.05, 1.0))), "hi": hi,
            "causal": rng.random() < 0.8}


def _spread(lo, hi, batch):
    """A length for each request between lo and hi, both of them met, in no order of size."""
    if batch == 1:
        return np.array([hi], np.int64)
    steps = (np.arange(batch) * 7919) % batch if batch % 7919 else np.arange(batch)
    return lo + (steps * (hi - lo)) // (batch - 1)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


# ---------------------------------------------------------------- inputs

def _logits(rows, vocab, flat, g, dev):
    """Logits as a head leaves them: a broad bulk, and a few dozen tokens far above it whose
    lead falls off (``flat`` of the lead is taken away)."""
    x = torch.randn(rows, vocab, generator=g, device=dev).mul_(2.2)
    n = min(vocab, 48)
    at = torch.randint(vocab, (rows, n), generator=g, device=dev)
    lead = torch.rand(rows, n, generator=g, device=dev).log_().neg_().mul_(3.0).add_(6.0).mul_(1.0 - flat)
    return x.scatter_add_(1, at, lead)


def _settings(case, count, g, dev):
    """The sampling settings of `count` requests: near the case's, no two requests alike."""
    near = torch.rand(count, generator=g, device=dev).mul_(0.1).add_(0.95)
    s = {"temperature": near * case["temperature"], "top_k": None, "top_p": None, "min_p": None}
    if case["top_k"]:
        s["top_k"] = (near * case["top_k"]).round().clamp_(min=1).int()
    if case["top_p"] < 1.0:
        s["top_p"] = (1.0 - near * (1.0 - case["top_p"])).contiguous()
    if case["min_p"]:
        s["min_p"] = near * case["min_p"]
    return s


def _offsets(draft_vocab, vocab, g, dev):
    """The offset table of a drafter that keeps draft_vocab of vocab tokens: id = i + d2t[i]."""
    if draft_vocab >= vocab:
        return None
    ids = torch.randperm(vocab, generator=g, device=dev)[:draft_vocab].sort().values
    return (ids - torch.arange(draft_vocab, device=dev)).int()


def _package():
    import drafting_eagle_draft_gb300 as pk
    return pk


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * int(seed) + 29)
    return {"sample": _prepare_sample, "verify": _prepare_verify, "attention": _prepare_attention}[case["op"]](case, g, dev)


def _prepare_sample(case, g, dev):
    R, V, per = case["rows"], case["vocab"], case["per"]
    s = {"case": case, "logits": _logits(R, V, case["flat"], g, dev).to(_dtype(case)),
         "how": _settings(case, (R + per - 1) // per, g, dev),
         "u": torch.rand(R, generator=g, device=dev), "d2t": _offsets(V, case["target"], g, dev),
         "token": torch.zeros(R, dtype=torch.int32, device=dev), "prob": torch.zeros(R, device=dev)}
    if own:
        s["struct"] = _package().sampling_struct(**s["how"], rows_per=per)
    return s


def _prepare_verify(case, g, dev):
    B, K, V, D = case["batch"], case["K"], case["vocab"], case["draft_vocab"]
    s = {"case": case, "how": _settings(case, B, g, dev), "d2t": _offsets(D, V, g, dev)}
    target = _logits(B * (K + 1), V, 0.0, g, dev)
    # the drafter's logits: the target's own at its tokens, and how far it is from it
    draft = target.view(B, K + 1, V)[:, :K].reshape(B * K, V)
    if s["d2t"] is not None:
        draft = draft[:, torch.arange(D, device=dev) + s["d2t"]]
    draft = draft + torch.randn(B * K, D, generator=g, device=dev).mul_(0.7)
    s["target"], s["draft"] = target.to(_dtype(case)), draft.contiguous()
    u = torch.rand(B * (2 * K + 1), generator=g, device=dev)
    s["u_draft"], s["u_accept"], s["u_bonus"] = u[:B * K], u[B * K:2 * B * K], u[2 * B * K:]
    s["accept"] = torch.zeros(B, dtype=torch.int32, device=dev)
    s["bonus"] = torch.zeros(B, dtype=torch.int32, device=dev)
    s["chance"] = torch.zeros(B, K, device=dev)
    if own:
        pk = _package()
        # the round's drafts, as the call before this one leaves them
        s["token"] = torch.zeros(B * K, dtype=torch.int32, device=dev)
        s["dist"] = None if case["greedy"] else pk.sample_dist(B * K, dev)
        how = {"temperature": torch.zeros(B, device=dev)} if case["greedy"] else s["how"]
        how = pk.sampling_struct(**how, rows_per=K)
        pk.peagle_sample(how, s["draft"], s["u_draft"], s["token"], d2t=s["d2t"], out_dist=s["dist"])
        s["struct"] = pk.sampling_struct(**s["how"], rows_per=K + 1)
        s["work"] = torch.empty(pk.peagle_verify_sample_workspace(B, K, V), dtype=torch.uint8, device=dev)
    elif case["greedy"]:
        s["index"] = s["draft"].argmax(-1)
    else:
        s["index"] = _pick(_weights(s["draft"], _of_rows(s["how"], K, B * K)), s["u_draft"])
    return s


def _prepare_attention(case, g, dev):
    B, K, nq, H, hd, P = (case[k] for k in ("batch", "K", "heads", "kv_heads", "head_dim", "prefix"))

    def rows(*shape):
        x = torch.randn(shape, generator=g, device=dev)
        channel = torch.ones(shape[-1], device=dev)
        channel[torch.randint(shape[-1], (4,), generator=g, device=dev)] = 4.0
        return x.mul_(channel).to(_dtype(case))

    lens = _spread(case["lo"], case["hi"], B)
    cap = int(lens.max()) + K + 5
    s = {"case": case, "prefix_k": rows(H, P + 3, hd), "prefix_v": rows(H, P + 3, hd),
         "k": rows(B, H, cap, hd), "v": rows(B, H, cap, hd),
         "prefix_len": torch.full((1,), P, dtype=torch.int32, device=dev),
         "lens": torch.from_numpy(lens.astype(np.int32)).to(dev),
         "q": torch.randn(B * K, nq, hd, generator=g, device=dev).to(_dtype(case)),
         "out": torch.zeros(B * K, nq, hd, dtype=_dtype(case), device=dev),
         "lse": torch.zeros(B * K, nq, device=dev),
         "slots": int(lens.max()) + (K if case["causal"] else 0)}
    if own:
        n = _package().peagle_decode_attention_shared_workspace(B, K, s["q"], s["prefix_k"], s["k"])
        s["work"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"sample": _run_sample, "verify": _run_verify, "attention": _run_attention}[s["case"]["op"]](s)


def _of_rows(how, per, rows):
    """The settings of each row: `per` rows in a row share a request's."""
    at = torch.arange(rows, device=how["temperature"].device) // per
    return {k: None if v is None else v[at] for k, v in how.items()}


def _weights(logits, how):
    """The kept tokens' exp((x - max) / temperature), zero elsewhere; in 64 bits, because the sums
    decide between neighbours."""
    x = logits.double()
    top = x.amax(-1, keepdim=True)
    w = ((x - top) / how["temperature"].double()[:, None]).exp_()
    if how["top_k"] is None and how["top_p"] is None:
        return w if how["min_p"] is None else w * (w >= how["min_p"].double()[:, None])
    order = x.sort(dim=-1, descending=True, stable=True).indices  # ties: the lowest index first
    del x
    s = w.gather(-1, order)
    keep = torch.ones_like(s, dtype=torch.bool)
    if how["top_k"] is not None:
        keep = torch.arange(s.shape[-1], device=s.device) < how["top_k"][:, None]
        s = s * keep
    if how["top_p"] is not None:
        before = s.cumsum(-1).sub_(s)
        keep &= before < how["top_p"].double()[:, None] * s.sum(-1, keepdim=True)
        keep[:, 0] = True
    if how["min_p"] is not None:
        keep &= s >= how["min_p"].double()[:, None]
    return w * torch.zeros_like(keep).scatter_(-1, order, keep)


def _pick(w, u):
    """The first token at which the weights' running sum passes u of the whole."""
    c = w.cumsum(-1)
    n = (c <= u.double()[:, None] * c[:, -1:]).sum(-1)
    return n.clamp_(max=w.shape[-1] - 1)


def _run_sample(s):
    c = s["case"]
    if own:
        _package().peagle_sample(s["struct"], s["logits"], s["u"], s["token"], d2t=s["d2t"], out_prob=s["prob"])
        return {"token": s["token"], "prob": s["prob"]}
    w = _weights(s["logits"], _of_rows(s["how"], c["per"], c["rows"]))
    i = _pick(w, s["u"])
    s["prob"].copy_(w.gather(-1, i[:, None])[:, 0] / w.sum(-1))
    s["token"].copy_(i if s["d2t"] is None else i + s["d2t"][i])
    return {"token": s["token"], "prob": s["prob"]}


def _run_verify(s):
    c = s["case"]
    B, K, V, D = c["batch"], c["K"], c["vocab"], c["draft_vocab"]
    if own:
        _package().peagle_verify_sample(
            B, K, s["token"], s["struct"], s["target"], s["u_accept"], s["u_bonus"], s["accept"], s["bonus"], s["work"],
            draft_logits=None if c["greedy"] else s["draft"], draft_dist=s["dist"], d2t=s["d2t"], out_accept_prob=s["chance"])
        return {"accept": s["accept"], "bonus": s["bonus"], "chance": s["chance"]}
    i = s["index"]  # of the drafts, in the drafter's vocabulary
    ids = torch.arange(D, device=i.device)
    if s["d2t"] is not None:
        ids = ids + s["d2t"]
    p = _weights(s["target"], _of_rows(s["how"], K + 1, B * (K + 1))).view(B, K + 1, V)
    p = p / p.sum(-1, keepdim=True)
    at = p[:, :K].gather(-1, ids[i].view(B, K, 1))[..., 0]
    if c["greedy"]:
        q = torch.zeros(B, K, D, dtype=torch.float64, device=i.device).scatter_(-1, i.view(B, K, 1), 1.0)
    else:
        q = _weights(s["draft"], _of_rows(s["how"], K, B * K)).view(B, K, D)
        q = q / q.sum(-1, keepdim=True)
    mine = q.gather(-1, i.view(B, K, 1))[..., 0]
    s["chance"].copy_((at / mine).clamp_(max=1.0))
    ok = s["u_accept"].view(B, K).double() * mine < at
    m = ok.int().cumprod(-1).sum(-1)
    rows = torch.arange(B, device=i.device)
    left = p[rows, m]
    taken = torch.where((m < K)[:, None], q[rows, m.clamp(max=K - 1)], 0.0)
    rest = left.scatter_add(-1, ids.expand(B, D), -taken).clamp_(min=0.0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, left)
    s["accept"].copy_(m)
    s["bonus"].copy_(_pick(rest, s["u_bonus"]))
    return {"accept": s["accept"], "bonus": s["bonus"], "chance": s["chance"]}


def _run_attention(s):
    c = s["case"]
    B, K, nq, H, hd, P, n = (c["batch"], c["K"], c["heads"], c["kv_heads"], c["head_dim"], c["prefix"], s["slots"])
    if own:
        _package().peagle_decode_attention_shared(
            B, K, s["q"], s["prefix_k"], s["prefix_v"], s["prefix_len"], s["k"], s["v"], s["lens"], s["out"], s["work"],
            out_lse=s["lse"], causal=c["causal"])
        return {"out": s["out"], "lse": s["lse"]}
    G, scale = nq // H, 1.0 / math.sqrt(hd)
    q = s["q"].float().view(B, K, H, G, hd)
    shared = q.permute(2, 0, 1, 3, 4).reshape(H, B * K * G, hd)
    a = torch.matmul(shared, s["prefix_k"][:, :P].float().transpose(-1, -2)).mul_(scale).view(H, B, K, G, P)
    mine = q.permute(0, 2, 1, 3, 4).reshape(B, H, K * G, hd)
    b = torch.matmul(mine, s["k"][:, :, :n].float().transpose(-1, -2)).mul_(scale).view(B, H, K, G, n)
    end = s["lens"][:, None] + (torch.arange(K, device=q.device) + 1 if c["causal"] else torch.zeros(K, device=q.device, dtype=torch.int64))
    unseen = torch.arange(n, device=q.device) >= end[..., None]
    b = b.masked_fill_(unseen[:, None, :, None, :], -math.inf).permute(1, 0, 2, 3, 4)  # as the prefix: heads first
    top = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
    a = a.sub_(top).exp_()
    b = (b - top).exp_()
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    out = torch.matmul(a.view(H, B * K * G, P), s["prefix_v"][:, :P].float()).view(H, B, K, G, hd)
    more = torch.matmul(b.permute(1, 0, 2, 3, 4).reshape(B, H, K * G, n), s["v"][:, :, :n].float())
    out = (out + more.view(B, H, K, G, hd).permute(1, 0, 2, 3, 4)) / total
    s["out"].copy_(out.permute(1, 2, 0, 3, 4).reshape(B * K, nq, hd))
    s["lse"].copy_((top + total.log()).squeeze(-1).permute(1, 2, 0, 3).reshape(B * K, nq))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        # a difference, a product, an exponential and a sum for each logit
        return {"bytes": n * _size(case) + 16 * case["rows"], "flops": 4 * n}
    if case["op"] == "verify":
        B, K, V, D = case["batch"], case["K"], case["vocab"], case["draft_vocab"]
        n = B * (K + 1) * V
        # the target's rows, and the one draft row that a request's first rejection asks for
        return {"bytes": n * _size(case) + (0 if case["greedy"] else B * D * 4) + B * (12 * K + 12),
                "flops": 4 * n + 6 * B * V}
    B, K, nq, H, hd, P = (case[k] for k in ("batch", "K", "heads", "kv_heads", "head_dim", "prefix"))
    lens = _spread(case["lo"], case["hi"], B)
    extra = K if case["causal"] else 0
    pairs = B * K * P + int(sum(K * n + extra * (extra + 1) // 2 for n in lens))
    slots = P + int(lens.sum()) + B * extra
    rows = B * K * nq
    return {"bytes": 2 * slots * H * hd * _size(case) + rows * (2 * hd * _size(case) + 4), "flops": 4 * hd * nq * pairs}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"sample": _exact_sample, "verify": _exact_verify, "attention": _exact_attention}[case["op"]](case, s)


def _exact_row(logits, how, r):
    """One row's distribution, the kept tokens in the order of their size."""
    x = logits.double()
    x, order = torch.sort(-x, stable=True)
    w = torch.exp((x[0] - x) / how["temperature"][r].double())
    n = w.numel()
    if how["top_k"] is not None:
        n = min(n, int(how["top_k"][r]))
    if how["top_p"] is not None:
        c = torch.cumsum(w[:n], 0)
        want = how["top_p"][r].double() * c[-1]
        n = min(n, int(torch.searchsorted(c, want.reshape(1))[0]) + 1)  # the first prefix that reaches it
    if how["min_p"] is not None:
        n = min(n, int((w >= how["min_p"][r].double()).sum()))
    p = torch.zeros_like(w)
    p[order[:n]] = w[:n] / w[:n].sum()
    return p


def _exact_pick(p, u):
    c = torch.cumsum(p, 0)
    return min(int(torch.searchsorted(c, (u.double() * c[-1]).reshape(1), right=True)[0]), p.numel() - 1)


def _exact_sample(case, s):
    out = []
    for r in range(case["rows"]):
        p = _exact_row(s["logits"][r], s["how"], r // case["per"])
        out.append(p[_exact_pick(p, s["u"][r])])
    return {"token": None, "prob": torch.stack(out)}


def _exact_verify(case, s):
    if own:
        return None  # the drafts' indices are inside the package's records
    B, K = case["batch"], case["K"]
    chance = torch.zeros(B, K, dtype=torch.float64)
    for b in range(B):
        for j in range(K):
            i = int(s["index"][b * K + j])
            token = i if s["d2t"] is None else i + int(s["d2t"][i])
            p = _exact_row(s["target"][b * (K + 1) + j], s["how"], b)[token]
            q = 1.0 if case["greedy"] else _exact_row(s["draft"][b * K + j], s["how"], b)[i]
            chance[b, j] = min(1.0, float(p / q))
    return {"accept": None, "bonus": None, "chance": chance}


def _exact_attention(case, s):
    B, K, nq, H, hd, P = (case[k] for k in ("batch", "K", "heads", "kv_heads", "head_dim", "prefix"))
    G = nq // H
    dev = s["q"].device
    out = torch.zeros(B, K, H, G, hd, dtype=torch.float64, device=dev)
    lse = torch.zeros(B, K, H, G, dtype=torch.float64, device=dev)
    q = s["q"].double().view(B, K, H, G, hd) / math.sqrt(hd)
    for h in range(H):
        pk, pv = s["prefix_k"][h, :P].double(), s["prefix_v"][h, :P].double()
        for b, n in enumerate(s["lens"].tolist()):
            e = n + K if case["causal"] else n
            k, v = torch.cat([pk, s["k"][b, h, :e].double()]), torch.cat([pv, s["v"][b, h, :e].double()])
            x = torch.einsum("jgd,td->jgt", q[b, :, h], k)
            if case["causal"]:
                at = torch.arange(P + e, device=dev) - P - n
                x[at[None, None].expand_as(x) > torch.arange(K, device=dev)[:, None, None]] = -math.inf
            lse[b, :, h] = torch.logsumexp(x, -1)
            out[b, :, h] = torch.einsum("jgt,td->jgd", torch.exp(x - lse[b, :, h][..., None]), v)
    return {"out": out.view(B * K, nq, hd), "lse": lse.view(B * K, nq)}
