"""The block step over the 8-bit cache: B masked positions of every sequence are rotated and attended to, the head
accepts a prefix of them, and what it accepted is appended, its count going from one call to the next on the GPU
(needs a GB300)."""
import numpy as np
import pytest
import torch

import oracle
from block_masked_token_gb300 import mars, packed
from packed_util import PAGE, f64, workspace
from parity_util import compare_head
from test_q8_gpu import check_chunk8, check_rotary, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch, B, heads", [(20, 16, (28, 4, 128)), (12, 4, (14, 2, 64)), (9, 8, (24, 1, 128))], ids=str)
def test_block_steps_from_one_graph(batch, B, heads):
    hq, hkv, d = heads
    hidden, vocab, tau, width, steps = 256, 512, 0.5, 12, 6
    g = torch.Generator().manual_seed(B)
    pages = batch * width
    table = torch.randperm(pages, generator=g).to(torch.int32).view(batch, width)
    pools = {c + "_pool": torch.full((pages, hkv, PAGE, d), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for c in "kv"}
    cache = {**pools, **{c + "_scale": torch.full((pages, hkv), 255, dtype=torch.uint8, device="cuda") for c in "kv"}}
    pool_args = [cache[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale")]
    freq, factor = packed.rotary_frequencies(d, scaling="base", stretch=2.0)
    freq, st = freq.cuda(), status()
    w = torch.randn(vocab, hidden, generator=g).to(torch.bfloat16)
    n, hint, T = batch * B, width * PAGE, table.cuda()
    cu = torch.arange(0, n + 1, B, dtype=torch.int32)
    qkv = torch.zeros(n, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    h, o = torch.zeros(n, hidden, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    lens, new = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda")
    count = torch.zeros_like(lens)
    tokens, p = torch.zeros(batch, B, dtype=torch.int32, device="cuda"), torch.zeros(batch, B, device="cuda")
    slots, C, W_ = torch.zeros(n, dtype=torch.int32, device="cuda"), cu.cuda(), w.cuda()
    ws = workspace(packed.OP_ATTN_CHUNK_Q8, batch, n, hq, hkv, d, hint)
    head_ws = torch.empty(mars.mars_workspace_bytes(mars.OP_HEAD_ACCEPT, batch, B, vocab=vocab), dtype=torch.uint8, device="cuda")

    # prompts of every length, from none on
    prompt = [(29 * i) % 70 for i in range(batch)]
    rows = torch.randn(sum(prompt), 2, hkv, d, generator=g).to(torch.bfloat16).cuda()
    packed.mars_kv_append_q8(rows[:, 0].contiguous(), rows[:, 1].contiguous(), torch.tensor(np.cumsum([0] + prompt), dtype=torch.int32).cuda(),
                             lens, T, *pool_args, new_lens=new, status=st)
    lens.copy_(new)

    def step():
        packed.mars_rotary(q, k, C, freq, q, k, seq_lens=lens, factor=factor, status=st)
        packed.mars_attn_chunk_q8(q, k, v, C, *pool_args, T, lens, hint, o, ws, status=st)
        mars.mars_head_accept(h, W_, batch, B, tau, tokens, p, count, head_ws, status=st)
        packed.mars_kv_append_q8(k, v, C, lens, T, *pool_args, counts=count, new_lens=new, slots=slots, status=st)
        lens.copy_(new)

    def fill():
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        # some positions sure of a word, the others of none
        sure = torch.rand(n, 1, generator=g) < 0.8
        words = w[torch.randint(vocab, (n,), generator=g)].float()
        h.copy_(torch.where(sure, words * 0.2, words * 1e-3))

    def host():
        return {name: t.cpu() for name, t in cache.items()}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = {name: t.clone() for name, t in cache.items()}
    with torch.cuda.stream(side):
        step()                                       # first calls set attributes up
    torch.cuda.synchronize()
    for name, t in keep.items():
        cache[name].view(torch.uint8).copy_(t.view(torch.uint8))
    lens.copy_(torch.tensor(prompt, dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = set()
    for _ in range(steps):
        fill()
        before, state = lens.cpu(), host()
        raw = {c: t.cpu().clone() for c, t in (("q", q), ("k", k))}
        o.fill_(7.0)
        slots.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        x = dict(n=n, lens=[B] * batch, cu=cu, old=before, table=table, fused=False, q=q.cpu(), k=k.cpu(), v=v.cpu(), **state)
        check_rotary(dict(n=n, cu=cu, **raw), (x["q"], x["k"]), before.tolist(), freq.cpu(), 7.0, factor=factor)
        check_chunk8(x, o)
        want = oracle.head_accept(f64(h), f64(w), batch, B, tau)
        compare_head(tokens.cpu().numpy(), p.cpu().numpy(), count.cpu().numpy(), *want, tau)
        accepted = count.tolist()
        seen.update(accepted)
        *want, wl, wslots = oracle.kv_append_q8(f64(x["k"]), f64(x["v"]), cu.numpy(), before.numpy(), table.numpy(), f64(state["k_pool"].float()),
                                                f64(state["v_pool"].float()), state["k_scale"].numpy(), state["v_scale"].numpy(),
                                                PAGE, accepted)
        np.testing.assert_array_equal(lens.cpu().numpy(), wl)
        np.testing.assert_array_equal(slots.cpu().numpy(), wslots)
        after = host()
        for c, i in (("k", 0), ("v", 1)):
            np.testing.assert_array_equal(after[c + "_scale"].numpy(), want[2 + i])
            np.testing.assert_array_equal(f64(after[c + "_pool"].float()), want[i])
    assert int(st.item()) == 0 and len(seen) > 2
