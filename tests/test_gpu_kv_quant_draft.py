"""Draft rows in the 8-bit cache that are dropped again: with the open block saved before and
restored after, the cache is bit for bit the one that never saw them."""
import numpy as np
import pytest
import torch

from pe_helpers import pk
from test_gpu_kv_quant import Cache, fresh, ints, queries, rows_like

pytestmark = pytest.mark.gpu


def committed(c, lens):
    """Codes of the committed slots and the scales of their blocks."""
    got = []
    for name in ("k", "v"):
        for b, n in enumerate(lens):
            got.append(c.t[name].view(torch.uint8)[:, b, :, :n].clone())
            got.append(c.t[name + "_scale"][:, b, :, :-(-n // c.block)].clone())
    return got


def equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
def test_dropped_drafts_leave_no_trace(hd, block, dtype):
    m = pk()
    L, B, H, cap, K = 2, 5, 3, 256, 6
    c, never, traced = (fresh(L, B, H, cap, hd, block) for _ in range(3))
    lens = [0, 1, block - 1, block, 53]
    prompt = [rows_like((L, B, 128, H, hd), i, dtype, 1.0) for i in (1, 2)]
    for x in (c, never, traced):
        m.peagle_append_kv_quant(x.kv, B, ints([0] * B), ints(lens), *prompt, 128)
    saved = torch.full((m.peagle_save_kv_quant_bytes(c.kv),), 0xff, dtype=torch.uint8, device="cuda")
    for step in range(8):
        sl = ints(lens)
        draft = [rows_like((L, B, K, H, hd), 10 + 2 * step + i, dtype, 1.0) for i in (0, 1)]
        for x in draft:
            x[:, :, K - 1, :, 5] = 3e4  # the last draft row is never accepted here
        accepted = [(step + b) % K for b in range(B)]
        m.peagle_save_kv_quant(c.kv, B, sl, saved)
        for x in (c, traced):
            for layer in range(L):
                m.peagle_append_kv_quant(x.kv, B, sl, None, draft[0][layer], draft[1][layer], K,
                                         layer=layer, n_extra=K, advance=False)
        if step % 2:
            m.peagle_restore_kv_quant(c.kv, B, sl, saved)
        else:
            for layer in range(L):
                m.peagle_restore_kv_quant(c.kv, B, sl, saved, layer=layer)
        assert equal(committed(c, lens), committed(never, lens))
        for x in (c, never, traced):
            m.peagle_append_kv_quant(x.kv, B, ints(lens), ints(accepted), *draft, K)
        lens = [a + n for a, n in zip(lens, accepted)]
        assert equal(committed(c, lens), committed(never, lens))
    assert not equal(committed(traced, lens), committed(never, lens))
    assert c.err() == 0 and never.err() == 0


def test_save_and_restore_touch_only_what_they_say():
    """One layer of several, fewer requests than the cache holds, lengths at a block's edge, at the
    capacity and out of range."""
    m = pk()
    L, B, H, hd, cap, block = 3, 6, 2, 64, 96, 32
    c = Cache(L, B, H, cap, hd, block, 5)
    lens = [0, 7, 32, 96, -1, 97]
    saved = torch.zeros(m.peagle_save_kv_quant_bytes(c.kv), dtype=torch.uint8, device="cuda")
    m.peagle_save_kv_quant(c.kv, B, ints(lens), saved, layer=1)
    assert c.err() == m.PEAGLE_DEV_KV_OVERFLOW
    codes = saved[:2 * L * B * H * block * hd].view(2, L, B, H, block, hd)
    scales = saved[codes.numel():].view(torch.float32).view(2, L, B, H)
    for i, name in enumerate("kv"):
        x = c.t[name].view(torch.uint8)
        assert torch.equal(codes[i, 1, 1, :, :7], x[1, 1, :, :7])
        assert torch.equal(scales[i, 1, 1], c.t[name + "_scale"][1, 1, :, 0])
    codes[:, 1, 1, :, :7] = 0
    assert not codes.any() and int((scales != 0).sum()) == 2 * H
    before = {k: t.clone() for k, t in c.t.items()}
    m.peagle_restore_kv_quant(c.kv, 4, ints(lens[:4]), saved, layer=1)
    assert c.err() == 0
    for name in "kv":
        x = before[name].view(torch.uint8)
        x[1, 1, :, :7] = 0
        assert torch.equal(c.t[name].view(torch.uint8), x)
        assert torch.equal(c.t[name + "_scale"], before[name + "_scale"])
    with pytest.raises(m.PeagleError):
        m.peagle_save_kv_quant(c.kv, B, ints(lens), saved[:-1])
    with pytest.raises(m.PeagleError):
        m.peagle_save_kv_quant(c.kv, B, ints(lens), saved.cpu())


def test_captured_rounds_with_drafts_that_are_dropped():
    """save, draft append, attention, restore, commit in one CUDA graph, against eager rounds of a
    cache that only sees what is accepted."""
    m = pk()
    L, B, H, hd, K, block, nq, cap = 1, 2, 2, 64, 5, 32, 8, 160
    c, e = fresh(L, B, H, cap, hd, block), fresh(L, B, H, cap, hd, block)
    rows = torch.zeros(2, L, B, K, H, hd, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B * K, nq, hd, dtype=torch.bfloat16, device="cuda")
    out, n, sl = torch.zeros_like(q), ints([0] * B), ints([0] * B)
    saved = torch.empty(m.peagle_save_kv_quant_bytes(c.kv), dtype=torch.uint8, device="cuda")
    work = torch.empty(m.peagle_decode_attention_quant_workspace(c.kv, B, K, nq), dtype=torch.uint8,
                       device="cuda")

    def step():
        m.peagle_save_kv_quant(c.kv, B, sl, saved)
        m.peagle_append_kv_quant(c.kv, B, sl, None, rows[0], rows[1], K, n_extra=K, advance=False)
        m.peagle_decode_attention_quant(c.kv, 0, B, K, nq, q, sl, out, work)
        m.peagle_restore_kv_quant(c.kv, B, sl, saved)
        m.peagle_append_kv_quant(c.kv, B, sl, n, rows[0], rows[1], K)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    sl.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    lens, esl = [0] * B, ints([0] * B)
    for i in range(20):
        rows.copy_(rows_like(tuple(rows.shape), 200 + i, "bf16", 1.0))
        rows[:, :, :, K - 1, :, 3] = 1e5
        accept = [i % K, (i + 2) % K]
        n.copy_(ints(accept))
        q.copy_(queries(B, K, nq, hd, "bf16", 300 + i, 5.0))
        g.replay()
        m.peagle_append_kv_quant(e.kv, B, esl, ints(accept), rows[0], rows[1], K)
        lens = [a + x for a, x in zip(lens, accept)]
        assert sl.tolist() == lens == esl.tolist()
        assert equal(committed(c, lens), committed(e, lens))
    assert c.err() == 0 and e.err() == 0 and np.isfinite(out.float().cpu().numpy()).all()
