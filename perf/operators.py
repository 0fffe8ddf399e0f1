"""The 8-bit drafter KV cache: what its operators compute, on which sizes they are measured.

A cache in 8 bits holds e4m3 codes [layer][request][kv head][slot][head_dim] and one fp32
scale for each block of slots of a (layer, request, kv head): a slot's value is code x scale.
The scale of a block is the smallest power of two s with |x| <= 448 s for every live value x
of the block (1 where all of them are zero).  Three operators share it:

  append     rows are quantised into the slots from a request's length on; the block that the
             rows start in is encoded again, with its earlier live rows, under its new scale
  read       slots are given back as bf16 or fp32 rows
  attention  K draft rows a request over the cached keys and values, for one layer

``run`` computes them in elementary torch operations, or, where ``own`` is set, through the
package's entry points.
"""
import math

import numpy as np
import torch

own = False

FP8 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 value


# ---------------------------------------------------------------- cases

def _attn(name, dtype, heads, kv_heads, head_dim, batch, K, lo, hi, block, window=0, causal=True):
    return {"name": name, "op": "attention", "dtype": dtype, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "batch": batch, "K": K, "lo": lo, "hi": hi, "block": block,
            "window": window, "causal": causal}


def _append(name, dtype, layers, kv_heads, head_dim, batch, n_lo, n_hi, lo, hi, block):
    return {"name": name, "op": "append", "dtype": dtype, "layers": layers, "kv_heads": kv_heads,
            "head_dim": head_dim, "batch": batch, "n_lo": n_lo, "n_hi": n_hi, "lo": lo, "hi": hi,
            "block": block}


def _read(name, dtype, layers, kv_heads, head_dim, batch, n_lo, n_hi, start, block):
    return {"name": name, "op": "read", "dtype": dtype, "layers": layers, "kv_heads": kv_heads,
            "head_dim": head_dim, "batch": batch, "n_lo": n_lo, "n_hi": n_hi, "start": start,
            "block": block}


def listed():
    return [
        # the tiny fp32 drafter's heads, one token over a short prompt: latency alone
        _attn("attn_token_tiny", "f32", 4, 2, 64, 1, 1, 128, 128, 16),
        # a draft pass of the H=2880 drafter, one request, K = 8 over 4096 slots
        _attn("attn_draft_b1", "bf16", 64, 8, 64, 1, 8, 4096, 4096, 32),
        # the same drafter at concurrency 2 with its 4096-position window
        _attn("attn_draft_b2_window", "bf16", 64, 8, 64, 2, 8, 8192, 10240, 32, window=4096),
        # the wide drafter, a ragged batch of 16
        _attn("attn_ragged_b16", "bf16", 32, 8, 128, 16, 5, 1024, 8192, 32),
        # a serving batch of the H=2880 drafter: many short contexts, 64 query rows a kv head
        _attn("attn_batch_b64", "bf16", 64, 8, 64, 64, 8, 301, 4099, 64),
        # long documents, one token each
        _attn("attn_long_token", "bf16", 32, 8, 128, 4, 1, 100003, 131071, 64),
        # fp32 queries over a committed prefix only, to be joined with other keys by its lse
        _attn("attn_prefix_f32", "f32", 32, 8, 128, 3, 5, 777, 5001, 128, causal=False),
        # a decode step's draft block written into every layer
        _append("append_step_b2", "bf16", 4, 8, 64, 2, 8, 8, 8191, 10240, 32),
        # the rows that a ragged batch of 16 accepted, kept in fp32 by the caller
        _append("append_ragged_b16", "f32", 4, 8, 128, 16, 1, 6, 1024, 8192, 64),
        # prompts of several requests quantised as a whole, out of a bf16 projection
        _append("append_prompt_b4", "bf16", 4, 8, 128, 4, 1001, 8192, 0, 0, 32),
        # a window of one request's slots read back into the 16-bit cache
        _read("read_window_b1", "bf16", 4, 8, 64, 1, 4096, 4096, 6150, 32),
        # parked requests brought back whole
        _read("read_all_b16", "bf16", 4, 8, 128, 16, 1024, 8192, 0, 32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "read"])
    head_dim = rng.choice([64, 128])
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "attention":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        K = rng.randint(1, min(16, 128 // group))
        batch = _log(rng, 1, 64)
        # cache bytes and products: at most about those of the largest listed cases
        most = min(4 * 8 * 100000 * 128 // (batch * kv_heads * head_dim),
                   int(2e10) // (4 * head_dim * kv_heads * group * batch * K))
        hi = _log(rng, 1, max(2, min(131072, most)))
        lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
        return {"op": op, "dtype": dtype, "heads": kv_heads * group, "kv_heads": kv_heads,
                "head_dim": head_dim, "batch": batch, "K": K, "lo": lo, "hi": hi, "block": block,
                "window": rng.choice([0, 0, _log(rng, 16, 8192)]), "causal": rng.random() < 0.75}
    layers = rng.randint(1, 6)
    batch = _log(rng, 1, 32)
    most = 4 * 8 * 128 * 4 * 8192 // (layers * kv_heads * head_dim * batch)
    n_hi = _log(rng, 1, max(2, min(16384, most)))
    n_lo = max(1, int(n_hi * rng.uniform(0.2, 1.0)))
    if op == "append":
        hi = rng.choice([0, _log(rng, 1, max(2, min(16384, most)))])
        return {"op": op, "dtype": dtype, "layers": layers, "kv_heads": kv_heads,
                "head_dim": head_dim, "batch": batch, "n_lo": n_lo, "n_hi": n_hi,
                "lo": int(hi * rng.uniform(0.2, 1.0)), "hi": hi, "block": block}
    return {"op": op, "dtype": dtype, "layers": layers, "kv_heads": kv_heads,
            "head_dim": head_dim, "batch": batch, "n_lo": n_lo, "n_hi": n_hi,
            "start": rng.choice([0, rng.randint(1, 4097)]), "block": block}


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


def _capacity(slots, block):
    """Whole blocks for the slots, and one to spare."""
    return (slots + block - 1) // block * block + block


# ---------------------------------------------------------------- inputs

def _scales(amax):
    """The smallest power of two s with amax <= 448 s, from amax's own bits; 1 for zero."""
    f, e = torch.frexp(amax)
    e = torch.where(f > 0.875, e - 8, e - 9).clamp(-40, 120)
    return torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), torch.ones_like(amax))


def _rows(shape, g, dev, dtype):
    """Keys or values as a drafter has them: N(0, 1) with a few large channels, and tokens whose
    size varies.  shape [..., slots, head_dim]."""
    x = torch.randn(shape, generator=g, device=dev)
    size = torch.randn(shape[:-1], generator=g, device=dev).mul_(0.6).exp_()
    channel = torch.ones(shape[-1], device=dev)
    channel[torch.randint(shape[-1], (4,), generator=g, device=dev)] = 6.0
    return (x * size[..., None] * channel).to(dtype)


def _cache(layers, batch, heads, capacity, head_dim, block, g, dev):
    """A cache in 8 bits, every block of it filled."""
    codes = torch.empty(layers, batch, heads, capacity, head_dim, dtype=FP8, device=dev)
    scale = torch.empty(layers, batch, heads, capacity // block, device=dev)
    for layer in range(layers):
        x = _rows((batch, heads, capacity, head_dim), g, dev, torch.float32)
        x = x.view(batch, heads, capacity // block, block * head_dim)
        s = _scales(x.abs().amax(-1))
        codes[layer] = (x / s[..., None]).view(batch, heads, capacity, head_dim).to(FP8)
        scale[layer] = s
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * int(seed) + 17)
    op, block, hd, H, B = case["op"], case["block"], case["head_dim"], case["kv_heads"], case["batch"]

    def ints(v):
        return torch.from_numpy(np.ascontiguousarray(v, np.int32)).to(dev)

    s = {"case": case}
    if op == "attention":
        lens = _spread(case["lo"], case["hi"], B)
        cap = _capacity(int(lens.max()) + case["K"], block)
        s["k"], s["k_scale"] = _cache(1, B, H, cap, hd, block, g, dev)
        s["v"], s["v_scale"] = _cache(1, B, H, cap, hd, block, g, dev)
        s["lens"] = ints(lens)
        s["q"] = torch.randn(B * case["K"], case["heads"], hd, generator=g, device=dev).to(_dtype(case))
        s["out"] = torch.zeros(B * case["K"], case["heads"], hd, dtype=_dtype(case), device=dev)
        s["lse"] = torch.zeros(B * case["K"], case["heads"], device=dev)
        s["slots"] = int(lens.max()) + (case["K"] if case["causal"] else 0)
    elif op == "append":
        L = case["layers"]
        lens, n = _spread(case["lo"], case["hi"], B), _spread(case["n_lo"], case["n_hi"], B)[::-1]
        cap = _capacity(int((lens + n).max()), block) + _capacity(int(n.max()), block)
        s["k"], s["k_scale"] = _cache(L, B, H, cap, hd, block, g, dev)
        s["v"], s["v_scale"] = _cache(L, B, H, cap, hd, block, g, dev)
        s["lens"], s["n"], s["n_max"] = ints(lens), ints(n), int(n.max())
        shape = (L, B, s["n_max"], H, hd)
        s["k_rows"] = _rows((L, B, H, s["n_max"], hd), g, dev, _dtype(case)).transpose(2, 3).contiguous()
        s["v_rows"] = _rows((L, B, H, s["n_max"], hd), g, dev, _dtype(case)).transpose(2, 3).contiguous()
        assert tuple(s["k_rows"].shape) == shape
    else:
        L = case["layers"]
        n = _spread(case["n_lo"], case["n_hi"], B)
        cap = _capacity(case["start"] + int(n.max()), block)
        s["k"], s["k_scale"] = _cache(L, B, H, cap, hd, block, g, dev)
        s["v"], s["v_scale"] = _cache(L, B, H, cap, hd, block, g, dev)
        s["n"], s["n_max"] = ints(n), int(n.max())
        s["starts"] = ints(np.full(B, case["start"]))
        # the 16-bit (or 32-bit) drafter cache that the slots go back to
        s["out_k"] = torch.zeros(L, B, H, s["n_max"], hd, dtype=_dtype(case), device=dev)
        s["out_v"] = torch.zeros(L, B, H, s["n_max"], hd, dtype=_dtype(case), device=dev)
    if own:
        import drafting_eagle_draft_gb300 as pk
        s["cache"] = pk.kv_quant_struct(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "attention":
            n = pk.peagle_decode_attention_quant_workspace(s["cache"], B, case["K"], case["heads"])
            s["work"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"attention": _attention, "append": _append_rows, "read": _read_slots}[s["case"]["op"]](s)


def _attention(s):
    c = s["case"]
    B, K, nq, H, hd = c["batch"], c["K"], c["heads"], c["kv_heads"], c["head_dim"]
    if own:
        import drafting_eagle_draft_gb300 as pk
        pk.peagle_decode_attention_quant(s["cache"], 0, B, K, nq, s["q"], s["lens"], s["out"], s["work"],
                                         out_lse=s["lse"], causal=c["causal"], window=c["window"])
        return {"out": s["out"], "lse": s["lse"]}
    G, n = nq // H, s["slots"]
    blocks = (n + c["block"] - 1) // c["block"]

    def values(codes, scale):
        x = codes[0, :, :, : blocks * c["block"]].float().view(B, H, blocks, c["block"], hd)
        return x.mul_(scale[0, :, :, :blocks, None, None]).view(B, H, blocks * c["block"], hd)[:, :, :n]

    q = s["q"].float().view(B, K, H, G, hd).transpose(1, 2).reshape(B, H, K * G, hd)
    score = torch.matmul(q, values(s["k"], s["k_scale"]).transpose(-1, -2)) * (1.0 / math.sqrt(hd))
    slot = torch.arange(n, device=q.device)
    at = s["lens"][:, None] + torch.arange(K, device=q.device)  # the rows' own positions
    end = at + 1 if c["causal"] else s["lens"][:, None].expand(B, K)
    seen = slot < end[..., None]
    if c["window"]:
        seen = seen & (slot > at[..., None] - c["window"])
    score = score.view(B, H, K, G, n).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(B, H, K * G, n), values(s["v"], s["v_scale"])).view(B, H, K, G, hd)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + total.log()).squeeze(-1)
    s["out"].copy_(out.transpose(1, 2).reshape(B * K, nq, hd))
    s["lse"].copy_(lse.transpose(1, 2).reshape(B * K, nq))
    return {"out": s["out"], "lse": s["lse"]}


def _append_rows(s):
    c = s["case"]
    B, block = c["batch"], c["block"]
    if own:
        import drafting_eagle_draft_gb300 as pk
        pk.peagle_append_kv_quant(s["cache"], B, s["lens"], s["n"], s["k_rows"], s["v_rows"], s["n_max"],
                                  advance=False)
        return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    dev = s["k"].device
    nb = (s["n_max"] + block - 1) // block + 1  # blocks that the rows of a request can touch
    lens, n = s["lens"].long(), s["n"].long()
    first = lens // block
    slot = first[:, None] * block + torch.arange(nb * block, device=dev)
    blk = first[:, None] + torch.arange(nb, device=dev)
    old = slot < lens[:, None]
    new = (slot >= lens[:, None]) & (slot < (lens + n)[:, None])
    touched = new.view(B, nb, block).any(-1)
    row = (slot - lens[:, None]).clamp(0, s["n_max"] - 1)
    b = torch.arange(B, device=dev)[:, None]

    def write(codes, scale, rows):
        bits = codes.view(torch.uint8)
        was = bits[:, b, :, slot]  # [B, slots, layers, heads, head_dim]
        was_scale = scale[:, b, :, blk]  # [B, blocks, layers, heads]
        L, H, hd = was.shape[2:]
        x = was.view(FP8).float().view(B, nb, block, L, H, hd).mul_(was_scale[:, :, None, :, :, None])
        x = torch.where(new[..., None, None, None], rows[:, b, row].float().permute(1, 2, 0, 3, 4),
                        x.view(B, nb * block, L, H, hd))
        live = (old | new)[..., None, None, None]
        amax = torch.where(live, x, torch.zeros_like(x)).abs().view(B, nb, block, L, H, hd).amax((2, 5))
        now = _scales(amax)
        code = (x.view(B, nb, block, L, H, hd) / now[:, :, None, :, :, None]).view(B, nb * block, L, H, hd).to(FP8)
        there = live & touched.repeat_interleave(block, 1)[..., None, None, None]
        bits[:, b, :, slot] = torch.where(there, code.view(torch.uint8), was)
        scale[:, b, :, blk] = torch.where(touched[..., None, None], now, was_scale)

    write(s["k"], s["k_scale"], s["k_rows"])
    write(s["v"], s["v_scale"], s["v_rows"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _read_slots(s):
    c = s["case"]
    B, block, n = c["batch"], c["block"], s["n_max"]
    if own:
        import drafting_eagle_draft_gb300 as pk
        pk.peagle_read_kv_quant(s["cache"], B, s["n"], s["out_k"].transpose(2, 3), s["out_v"].transpose(2, 3), n,
                                starts=s["starts"])
        return {"k": s["out_k"], "v": s["out_v"]}
    t = torch.arange(n, device=s["k"].device)
    slot = s["starts"].long()[:, None] + t
    inside = (t < s["n"][:, None])[:, None, :, None]
    b = torch.arange(B, device=s["k"].device)[:, None]

    def values(codes, scale, out):
        x = codes.view(torch.uint8)[:, b, :, slot].view(FP8).float()  # [B, n, layers, heads, head_dim]
        x.mul_(scale[:, b, :, slot // block][..., None])
        out.copy_(torch.where(inside, x.permute(2, 0, 3, 1, 4), out))

    values(s["k"], s["k_scale"], s["out_k"])
    values(s["v"], s["v_scale"], s["out_v"])
    return {"k": s["out_k"], "v": s["out_v"]}


# ---------------------------------------------------------------- what a pass cannot do without

def _seen(case):
    """(slots that some row of a request sees, (row, slot) pairs), over the requests."""
    slots = pairs = 0
    for n in _spread(case["lo"], case["hi"], case["batch"]):
        lo, hi = 1 << 60, 0
        for j in range(case["K"]):
            end = int(n) + j + 1 if case["causal"] else int(n)
            begin = max(0, int(n) + j - case["window"] + 1) if case["window"] else 0
            if end > begin:
                pairs += end - begin
                lo, hi = min(lo, begin), max(hi, end)
        slots += max(0, hi - lo)
    return slots, pairs


def work(case):
    hd, H, B, block = case["head_dim"], case["kv_heads"], case["batch"], case["block"]
    if case["op"] == "attention":
        slots, pairs = _seen(case)
        G = case["heads"] // H
        rows = B * case["K"] * case["heads"]
        return {"bytes": slots * H * (2 * hd + 8 / block) + rows * (2 * hd * _size(case) + 4) + 4 * B,
                "flops": 4 * hd * pairs * H * G}
    if case["op"] == "append":
        lens, n = _spread(case["lo"], case["hi"], B), _spread(case["n_lo"], case["n_hi"], B)[::-1]
        blocks = int(np.sum((lens + n + block - 1) // block - lens // block))
        units = 2 * case["layers"] * H
        # the new rows once in and once out as codes, the earlier codes of the first block in
        return {"bytes": units * (int(n.sum()) * hd * (_size(case) + 1) + int((lens % block).sum()) * hd + 4 * blocks),
                "flops": units * 3 * int(n.sum()) * hd}
    n = int(_spread(case["n_lo"], case["n_hi"], B).sum())
    units = 2 * case["layers"] * H
    return {"bytes": units * n * (hd * (1 + _size(case)) + 4 / block), "flops": units * n * hd}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    dev = s["k"].device
    with torch.no_grad():
        return {"attention": _exact_attention, "append": _exact_append, "read": _exact_read}[case["op"]](case, s, dev)


def _value64(s, which, layer, b, h, lo, hi):
    block = s["case"]["block"]
    scale = s[which + "_scale"][layer, b, h].double()
    return s[which][layer, b, h, lo:hi].double() * scale[torch.arange(lo, hi, device=scale.device) // block][:, None]


def _exact_attention(case, s, dev):
    B, K, nq, H, hd = case["batch"], case["K"], case["heads"], case["kv_heads"], case["head_dim"]
    G = nq // H
    out = torch.zeros(B, K, H, G, hd, dtype=torch.float64, device=dev)
    lse = torch.full((B, K, H, G), -math.inf, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["lens"].tolist()):
        q = s["q"].double().view(B, K, H, G, hd)[b]
        last = n + K if case["causal"] else n
        low = max(0, n - case["window"] + 1) if case["window"] else 0
        if last <= low:
            continue
        for h in range(H):
            k, v = _value64(s, "k", 0, b, h, low, last), _value64(s, "v", 0, b, h, low, last)
            score = torch.einsum("jgd,td->jgt", q[:, h], k) / math.sqrt(hd)
            for j in range(K):
                e = n + j + 1 if case["causal"] else n
                w = max(0, n + j - case["window"] + 1) if case["window"] else 0
                if e <= w:
                    continue
                x = score[j, :, w - low:e - low]
                lse[b, j, h] = torch.logsumexp(x, -1)
                out[b, j, h] = torch.exp(x - lse[b, j, h][:, None]) @ v[w - low:e - low]
    return {"out": out.view(B * K, nq, hd), "lse": lse.view(B * K, nq)}


def _power64(e):
    """2^e for whole e, as a double's own exponent field (pow and log2 are off by an ulp)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3_64(x):
    """The nearest e4m3 value (ties to the even one), in 64 bits: three bits after the leading
    one, and no exponent below 2^-6."""
    step = _power64(torch.frexp(x.abs().clamp_min(2.0 ** -6)).exponent - 4)
    return torch.round(x / step) * step


def _scale64(amax):
    """The smallest power of two s with amax <= 448 s, tried from a smaller one upwards."""
    e = torch.floor(torch.log2(amax.clamp_min(1e-300) / TOP)).long() - 1
    for _ in range(3):
        e = torch.where(amax > TOP * _power64(e), e + 1, e)
    return torch.where(amax > 0, _power64(e.clamp(-40, 120)), torch.ones_like(amax))


def _exact_append(case, s, dev):
    block, hd = case["block"], case["head_dim"]
    got = {}
    for which in ("k", "v"):
        codes, scale = s[which].double(), s[which + "_scale"].double()
        for b, (at, n) in enumerate(zip(s["lens"].tolist(), s["n"].tolist())):
            rows = s[which + "_rows"][:, b, :n].double().transpose(1, 2)  # [layers, heads, n, head_dim]
            t = at
            while t < at + n:
                i = t // block
                end = min(at + n, (i + 1) * block)
                before = codes[:, b, :, i * block:t] * scale[:, b, :, i, None, None]
                x = torch.cat([before, rows[:, :, t - at:end - at]], 2)
                if t == i * block and (end - t) == block and n > 4 * block:
                    # whole blocks from here on: all of them in one go
                    m = (at + n - t) // block
                    x = rows[:, :, t - at:t - at + m * block].reshape(rows.shape[0], rows.shape[1], m, block * hd)
                else:
                    m = 1
                    x = x.reshape(x.shape[0], x.shape[1], 1, -1)
                amax = x.abs().amax(-1)
                now = _scale64(amax)
                y = _e4m3_64(x / now[..., None]).reshape(x.shape[0], x.shape[1], -1, hd)
                codes[:, b, :, i * block:i * block + y.shape[2]] = y
                scale[:, b, :, i:i + m] = now
                t = i * block + m * block if m > 1 else end
        got[which], got[which + "_scale"] = codes, scale
    return got


def _exact_read(case, s, dev):
    got = {}
    for which in ("k", "v"):
        out = s["out_" + which].double()
        scale = s[which + "_scale"].double()
        for b, (at, n) in enumerate(zip(s["starts"].tolist(), s["n"].tolist())):
            of = torch.arange(at, at + n, device=dev) // case["block"]
            out[:, b, :, :n] = s[which][:, b, :, at:at + n].double() * scale[:, b][:, :, of][..., None]
        got[which] = out
    return got
