"""Packed prompts, chunks over the paged cache and the K/V append against the fp64 oracle
(needs a GB300). Bounds are elementwise, from the error model of parity_util and packed_util."""
import numpy as np
import pytest
import torch

import oracle
from block_masked_token_gb300 import mars, packed
from packed_util import (LSE_TOL, PAGE, causal_weights, cuda, f64, gradient_bounds, make,
                         output_bound, run_chunk, run_grad, run_packed, workspace)
from parity_util import assert_within_bound

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (7, 1, 128), (2, 2, 128), (14, 2, 64)]
LENS = [[1], [0, 1, 0, 2], [127, 128, 129], [19, 0, 300, 5], [513], [17, 18, 19, 36, 37]]


def check_packed(x, o, lse, fill=7.0, scale=None):
    ref, ref_lse = oracle.attn_packed(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["cu"].numpy(), scale)
    o, lse, cu = f64(o), f64(lse), x["cu"].tolist()
    g = x["q"].shape[1] // x["k"].shape[1]
    for a, b in zip(cu, cu[1:]):
        for h in range(x["q"].shape[1] if b > a else 0):
            P = causal_weights(f64(x["q"][a:b, h]), f64(x["k"][a:b, h // g]), scale)
            assert_within_bound(o[a:b, h], ref[a:b, h],
                                output_bound(P, f64(x["v"][a:b, h // g]), ref[a:b, h]), f"o rows {a}:{b} head {h}")
    live = ~np.isnan(ref_lse)
    assert np.abs(lse[live] - ref_lse[live]).max(initial=0.0) <= LSE_TOL
    # rows outside every sequence are left as they were
    outside = np.ones(x["n"], dtype=bool)
    outside[cu[0]:cu[-1]] = False
    assert (o[outside] == fill).all() and (lse[:, outside] == fill).all()


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_packed_matches_oracle(lens, heads):
    x = make(lens, *heads, seed=len(lens), tail=3, fused=heads[0] != 4)
    o, lse, st = run_packed(cuda(x))
    assert st == 0
    check_packed(x, o, lse)


@pytest.mark.parametrize("heads", [(130, 1, 64), (96, 1, 64), (128, 1, 64), (5, 5, 64)], ids=str)
def test_packed_group_sizes(heads):
    x = make([40, 3], *heads, seed=5)
    o, lse, st = run_packed(cuda(x))
    assert st == 0
    check_packed(x, o, lse)


# Many rows: two row tiles per item, several items per SM and items divided among SMs.
MANY = [([301, 40, 0, 517, 18, 19, 203, 37, 90, 200], (28, 4, 128)),
        ([600, 1, 35, 36, 37, 0, 513, 300, 128, 127, 129, 400, 250, 77, 150], (14, 2, 64)),
        ([1400], (28, 4, 128)), ([18] * 90, (28, 4, 128)), ([2000, 700], (4, 4, 64)),
        ([(331 * i) % 500 + 40 for i in range(22)], (28, 4, 128)),
        ([(97 * i) % 300 for i in range(60)], (28, 4, 64))]


@pytest.mark.parametrize("lens, heads", MANY, ids=str)
def test_packed_many_rows(lens, heads):
    x = make(lens, *heads, seed=31, tail=5, lead=1)
    o, lse, st = run_packed(cuda(x))
    assert st == 0
    check_packed(x, o, lse)
    again, lse2, _ = run_packed(cuda(x))
    assert same(o, again) and same(lse, lse2)


def test_packed_many_rows_of_more_sequences_than_a_ctas_threads():
    x = make([(i * 11) % 67 for i in range(500)], 14, 2, 64, seed=33, tail=2)
    o, lse, st = run_packed(cuda(x))
    assert st == 0
    check_packed(x, o, lse)


def test_packed_many_sequences_and_leading_rows():
    x = make([(i * 7) % 23 for i in range(75)], 4, 2, 64, seed=6, lead=5, tail=4)
    o, lse, st = run_packed(cuda(x))
    assert st == 0
    check_packed(x, o, lse)


def test_packed_scale_and_large_scores():
    """Scores of some tens: the running maximum has to be raised along a row."""
    x = make([200, 90], 4, 2, 64, seed=7)
    x["qkv"].mul_(2.0)
    o, lse, st = run_packed(cuda(x), scale=0.25)
    assert st == 0
    ref, _ = oracle.attn_packed(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["cu"].numpy(), 0.25)
    # scores are 8 times those of the model's inputs, and so is its upstream error of a weight,
    # 2^-14: the weights' sum of absolute errors is then at most 8 * 2^-14 * 2 max|v|
    slack = 16 * 2.0 ** -14 * np.abs(f64(x["v"])).max()
    o, cu = f64(o), x["cu"].tolist()
    for a, b in zip(cu, cu[1:]):
        for h in range(4):
            P = causal_weights(f64(x["q"][a:b, h]), f64(x["k"][a:b, h // 2]), 0.25)
            assert_within_bound(o[a:b, h], ref[a:b, h],
                                output_bound(P, f64(x["v"][a:b, h // 2]), ref[a:b, h]) + slack, "o")


def same(a, b):
    return torch.equal(a.cpu(), b.cpu())


def test_packed_other_rows_have_no_effect():
    """NaN and infinities in another sequence and behind the last one stay there."""
    x = make([70, 30, 150], 14, 2, 64, seed=8, tail=60)
    o, lse, _ = run_packed(cuda(x))
    x["qkv"][70:100] = float("nan")
    x["qkv"][250:] = float("inf")
    o2, lse2, st = run_packed(cuda(x))
    assert st == 0
    for rows in (slice(0, 70), slice(100, 250)):
        assert same(o[rows], o2[rows]) and same(lse[:, rows], lse2[:, rows])


def test_packed_later_keys_with_nan_scores_are_masked():
    x = make([100], 2, 1, 64, seed=9)
    o, lse, _ = run_packed(cuda(x))
    x["k"][60:] = float("nan")
    o2, lse2, _ = run_packed(cuda(x))
    assert same(o[:60], o2[:60]) and same(lse[:, :60], lse2[:, :60])


@pytest.mark.parametrize("cu, want", [([0, 40, 30, 90], [0, 40, 40, 90]),
                                      ([-5, 20, 200, 90], [0, 20, 90, 90]),
                                      ([0, 10, 50, 2000000000], [0, 10, 50, 90])])
def test_packed_bad_boundaries_are_cut(cu, want):
    x = make([20, 20, 50], 4, 2, 64, seed=10)
    x["cu"] = torch.tensor(cu, dtype=torch.int32)
    o, lse, st = run_packed(cuda(x))
    assert st == mars.ST_BADSEQ
    x["cu"] = torch.tensor(want, dtype=torch.int32)
    o2, lse2, st = run_packed(cuda(x))
    assert st == 0 and same(o, o2) and same(lse, lse2)


# ----------------------------------------------------------------------------- gradient

def check_grad(x, dq, dk, dv, fill=7.0):
    got, cu = {"q": f64(dq), "k": f64(dk), "v": f64(dv)}, x["cu"].tolist()
    ref = oracle.attn_packed_grad(*(f64(x[c]) for c in ("q", "k", "v", "do")), x["cu"].numpy())
    g = x["q"].shape[1] // x["k"].shape[1]
    for a, b in zip(cu, cu[1:]):
        for u in range(x["k"].shape[1] if b > a else 0):
            qs, k, v = gradient_bounds(x, a, b, u)
            np.testing.assert_allclose(k[0], ref[1][a:b, u], atol=1e-9)
            for i, (r, e) in enumerate(qs):
                assert_within_bound(got["q"][a:b, u * g + i], r, e, f"dq rows {a}:{b} head {u * g + i}")
            assert_within_bound(got["k"][a:b, u], *k, f"dk rows {a}:{b} head {u}")
            assert_within_bound(got["v"][a:b, u], *v, f"dv rows {a}:{b} head {u}")
    outside = np.ones(x["n"], dtype=bool)
    outside[cu[0]:cu[-1]] = False
    assert all((t[outside] == fill).all() for t in got.values())


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_gradient_matches_oracle(lens, heads):
    x = make(lens, *heads, seed=len(lens), tail=3, lead=2, fused=heads[0] != 4)
    y = cuda(x)
    o, lse, _ = run_packed(y)
    dq, dk, dv, st = run_grad(y, o, lse, y["do"], wide=heads[0] != 4)
    assert st == 0
    check_grad(x, dq, dk, dv)


def test_gradient_without_splits():
    """Enough key tiles that one item takes every query head of its KV head."""
    x = make([(i * 5) % 37 for i in range(80)], 16, 8, 64, seed=21)
    y = cuda(x)
    o, lse, _ = run_packed(y)
    dq, dk, dv, st = run_grad(y, o, lse, y["do"])
    assert st == 0
    check_grad(x, dq, dk, dv)


# Items divided among several CTAs, more heads than a block of prep takes, more sequences than
# the plan's CTA has threads.
GRAD_MANY = [([1500], (28, 4, 128)), ([700, 0, 301, 65], (14, 2, 64)), ([130, 40], (130, 2, 64)),
             ([(i * 11) % 67 for i in range(600)], (4, 2, 64))]


@pytest.mark.parametrize("lens, heads", GRAD_MANY, ids=["one", "few", "heads", "sequences"])
def test_gradient_of_many_rows(lens, heads):
    x = make(lens, *heads, seed=34, tail=3, lead=1)
    y = cuda(x)
    o, lse, _ = run_packed(y)
    dq, dk, dv, st = run_grad(y, o, lse, y["do"])
    assert st == 0
    check_grad(x, dq, dk, dv)
    again = run_grad(y, o, lse, y["do"])
    assert all(same(a, b) for a, b in zip((dq, dk, dv), again))


def test_training_steps_at_once_on_two_streams():
    """Calls with workspaces of their own do not disturb one another."""
    xs = [make([600, 90], 28, 4, 128, seed=35), make([40, 333, 7], 14, 2, 64, seed=36)]
    ys = [cuda(x) for x in xs]
    want = []
    for y in ys:
        o, lse, _ = run_packed(y)
        want.append([o, lse, *run_grad(y, o, lse, y["do"])[:3]])
    streams = [torch.cuda.Stream() for _ in ys]
    got = []
    for y in ys:
        n, hq, d = y["q"].shape
        b, hkv = len(y["cu"]) - 1, y["k"].shape[1]
        got.append([torch.full_like(y["do"], 7.0), torch.full((hq, n), 7.0, device="cuda"),
                    *torch.full((n, hq + 2 * hkv, d), 7.0, dtype=torch.bfloat16,
                                device="cuda").split([hq, hkv, hkv], dim=1),
                    workspace(packed.OP_ATTN_PACKED, b, n, hq, hkv, d),
                    workspace(packed.OP_ATTN_PACKED_GRAD, b, n, hq, hkv, d)])
    torch.cuda.synchronize()
    for _ in range(10):
        for y, g, stream in zip(ys, got, streams):
            o, lse, dq, dk, dv, ws, ws2 = g
            with torch.cuda.stream(stream):
                packed.mars_attn_packed(y["q"], y["k"], y["v"], y["cu"], o, ws, lse=lse)
                packed.mars_attn_packed_grad(y["q"], y["k"], y["v"], o, y["do"], lse, y["cu"], dq,
                                             dk, dv, ws2)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(same(a, b) for a, b in zip(w, g))


def test_gradient_of_single_tokens_is_exact():
    """One key: its weight is 1 whatever the score."""
    x = make([1] * 9, 4, 2, 64, seed=22)
    y = cuda(x)
    o, lse, _ = run_packed(y)
    dq, dk, dv, _ = run_grad(y, o, lse, y["do"])
    assert (dq == 0).all() and (dk == 0).all()
    assert same(dv, x["do"].float().view(9, 2, 2, 64).sum(2).to(torch.bfloat16))


def test_gradient_other_rows_have_no_effect_and_runs_agree():
    x = make([70, 30, 150], 14, 2, 64, seed=8, tail=60)
    y = cuda(x)
    o, lse, _ = run_packed(y)
    first = run_grad(y, o, lse, y["do"], fill=0.0)
    again = run_grad(y, o, lse, y["do"], fill=0.0)
    assert all(same(a, b) for a, b in zip(first[:3], again[:3]))
    for rows, bad in ((slice(70, 100), float("nan")), (slice(250, None), float("inf"))):
        y["qkv"][rows] = bad
        y["do"][rows] = bad
        o[rows] = bad
        lse[:, rows] = bad
    got = run_grad(y, o, lse, y["do"], fill=0.0)
    for a, b in zip(first[:3], got[:3]):
        assert same(a[:70], b[:70]) and same(a[100:250], b[100:250])


def test_gradient_bad_boundaries_are_cut():
    x = make([20, 20, 50], 4, 2, 64, seed=10)
    y = cuda(x)
    got = []
    for cu in ([0, 40, 30, 2000000], [0, 40, 40, 90]):
        y["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse, _ = run_packed(y)
        got.append(run_grad(y, o, lse, y["do"]))
    assert got[0][3] == mars.ST_BADSEQ and got[1][3] == 0
    assert all(same(a, b) for a, b in zip(got[0][:3], got[1][:3]))


def test_training_step_in_a_graph_and_on_another_stream():
    x = make([200, 1, 77], 14, 2, 64, seed=23)
    y = cuda(x)
    want_o, want_lse, _ = run_packed(y)
    want = run_grad(y, want_o, want_lse, y["do"], wide=False)[:3]
    o, lse = torch.zeros_like(want_o), torch.zeros_like(want_lse)
    out = [torch.zeros_like(t) for t in want]
    wf = workspace(packed.OP_ATTN_PACKED, 3, x["n"], 14, 2, 64)
    wg = workspace(packed.OP_ATTN_PACKED_GRAD, 3, x["n"], 14, 2, 64)

    def step(stream=None):
        packed.mars_attn_packed(y["q"], y["k"], y["v"], y["cu"], o, wf, lse=lse, stream=stream)
        packed.mars_attn_packed_grad(y["q"], y["k"], y["v"], o, y["do"], lse, y["cu"], *out, wg,
                                     stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(same(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (o, lse, *out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(o, want_o) and all(same(a, b) for a, b in zip(out, want))


# ------------------------------------------------------------------------------- chunks

def check_chunk(x, o, mapped=None):
    table = x["table"].numpy()
    ref = oracle.attn_chunk(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["cu"].numpy(),
                            f64(x["k_pool"]), f64(x["v_pool"]), table, x["old"].numpy(), PAGE)
    o, cu = f64(o), x["cu"].tolist()
    hq, hkv = x["q"].shape[1], x["k"].shape[1]
    kp, vp = f64(x["k_pool"]), f64(x["v_pool"])
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        pos = [(table[s, p // PAGE], p % PAGE) for p in range(int(x["old"][s]))]
        pos = [(e, c) for e, c in pos if 0 <= e < len(kp)]
        for h in range(hq if b > a else 0):
            u = h // (hq // hkv)
            K = np.concatenate([np.array([kp[e, u, c] for e, c in pos]).reshape(-1, kp.shape[-1]), f64(x["k"][a:b, u])])
            V = np.concatenate([np.array([vp[e, u, c] for e, c in pos]).reshape(-1, kp.shape[-1]), f64(x["v"][a:b, u])])
            P = causal_weights(f64(x["q"][a:b, h]), K)
            assert_within_bound(o[a:b, h], ref[a:b, h], output_bound(P, V, ref[a:b, h]), f"seq {s} head {h}")
    assert (o[cu[-1]:] == 7.0).all()


CHUNKS = [([1], [50]), ([1], [0]), ([1, 1, 1], [128, 1, 2300]), ([5, 0, 140, 1], [0, 77, 129, 513]),
          ([130], [1000]), ([19, 1], [127, 15]), ([1], [5000])]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lens, old", CHUNKS, ids=str)
def test_chunk_matches_oracle(lens, old, heads):
    x = make(lens, *heads, seed=sum(old), old=old, tail=2, fused=heads[0] != 4)
    # free slots of the pages hold NaN, as memory that nothing wrote may
    for s, p in enumerate(old):
        for c in range(p, -(-(p + lens[s]) // PAGE) * PAGE):
            x["k_pool"][x["table"][s, c // PAGE], :, c % PAGE] = float("nan")
            x["v_pool"][x["table"][s, c // PAGE], :, c % PAGE] = float("nan")
    x["k_pool"][x["unused"].long()] = float("nan")
    x["v_pool"][x["unused"].long()] = float("nan")
    o, st = run_chunk(cuda(x))
    assert st == 0
    check_chunk(x, o)


@pytest.mark.parametrize("lens, old, heads", [
    ([301, 40, 0, 217, 18, 1, 203, 37, 590], [300, 0, 77, 1000, 513, 129, 5, 700, 16], (28, 4, 128)),
    ([600, 1, 35, 36, 37, 0, 513, 300, 1, 127, 129, 400, 250, 77, 150],
     [0, 900, 64, 1, 2000, 9, 128, 130, 3000, 40, 0, 15, 16, 17, 250], (14, 2, 64)),
    ([1, 700, 1, 1], [4000, 1500, 17, 900], (28, 4, 128)), ([1] * 64, list(range(0, 1600, 25)), (28, 4, 128)),
    ([(331 * i) % 300 + 20 for i in range(28)], [(217 * i) % 900 for i in range(28)], (28, 4, 128))],
    ids=["ragged128", "ragged64", "mixed", "tokens", "whole"])
def test_chunk_many_rows(lens, old, heads):
    x = make(lens, *heads, seed=32, old=old, tail=3)
    y = cuda(x)
    o, st = run_chunk(y)
    assert st == 0
    check_chunk(x, o)
    for _ in range(20):                   # back to back, with different neighbours in time
        again, st = run_chunk(y)
        assert st == 0 and same(o, again)


@pytest.mark.parametrize("hint", [0, 100, 100000])
def test_chunk_hint_only_sizes_the_splits(hint):
    x = make([3, 1], 14, 2, 64, seed=3, old=[2000, 1300])
    o, st = run_chunk(cuda(x), hint=hint)
    assert st == 0
    check_chunk(x, o)


def test_chunk_unmapped_pages_are_skipped():
    x = make([4, 2], 4, 2, 64, seed=4, old=[200, 300])
    x["table"][0, 3] = -1
    x["table"][1, 0] = 1 << 20
    x["v_pool"][0] = float("nan") if 0 in x["unused"].tolist() else x["v_pool"][0]
    o, st = run_chunk(cuda(x))
    assert st == mars.ST_NOPAGE
    check_chunk(x, o)


def test_chunk_without_a_mapped_page_and_cut_lengths():
    x = make([2, 3], 4, 2, 64, seed=5, old=[40, 30])
    x["table"][:] = -1
    o, st = run_chunk(cuda(x))
    assert st == mars.ST_NOPAGE
    check_chunk(x, o)
    x = make([2, 3], 4, 2, 64, seed=5, old=[40, 30])
    y = cuda(x)
    y["old"] = torch.tensor([-3, 2000000000], dtype=torch.int32, device="cuda")
    y["table"][1] = y["table"][1].clamp(min=0)
    o, st = run_chunk(y, hint=100)
    x["old"] = torch.tensor([0, x["table"].shape[1] * PAGE], dtype=torch.int32)
    x["table"][1] = x["table"][1].clamp(min=0)
    assert st == mars.ST_OVERFLOW
    check_chunk(x, o)


def test_chunk_empty_pool():
    x = make([20, 1], 4, 2, 64, seed=6, old=[0, 0])
    y = cuda(x)
    y["k_pool"], y["v_pool"] = y["k_pool"][:0], y["v_pool"][:0]
    o, st = run_chunk(y)
    assert st == 0
    check_chunk(x, o)


# ------------------------------------------------------------------------------- append

def run_append(y, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.full_like(y["old"], -9)
    slots = torch.full((y["n"],), -9, dtype=torch.int32, device="cuda")
    packed.mars_kv_append(y["k"], y["v"], y["cu"], y["old"], y["table"], y["k_pool"], y["v_pool"],
                        new_lens=lens, slots=slots, status=st, **kw)
    torch.cuda.synchronize()
    return lens, slots, int(st.item())


@pytest.mark.parametrize("heads", [(4, 2, 64), (7, 1, 128), (10, 5, 64)], ids=str)
@pytest.mark.parametrize("lens, old", [([1], [50]), ([40, 0, 17, 1], [0, 31, 15, 16]), ([300, 16], [7, 0])], ids=str)
@pytest.mark.parametrize("hole", [None, 0, 1])
def test_append_matches_oracle(lens, old, heads, hole):
    x = make(lens, *heads, seed=1, old=old, tail=3)
    if hole is not None and hole < x["table"].shape[1]:
        x["table"][0, hole] = -1
    y = cuda(x)
    got_lens, slots, st = run_append(y)
    kp, vp, want_lens, want_slots = oracle.kv_append(
        f64(x["k"]), f64(x["v"]), x["cu"].numpy(), x["old"].numpy(), x["table"].numpy(),
        f64(x["k_pool"]), f64(x["v_pool"]), PAGE)
    assert (f64(y["k_pool"]) == kp).all() and (f64(y["v_pool"]) == vp).all()
    assert (got_lens.cpu().numpy() == want_lens).all()
    n = int(x["cu"][-1])
    assert (slots[:n].cpu().numpy() == want_slots[:n]).all() and (slots[n:] == -9).all()
    assert st == (0 if want_lens.sum() == sum(old) + sum(lens) else mars.ST_NOPAGE)


def test_append_past_the_table_and_negative_length():
    x = make([40, 20], 4, 2, 64, seed=2, old=[10, 5])
    x["table"] = x["table"][:, :2].contiguous()
    y = cuda(x)
    y["old"][1] = -1
    before = y["k_pool"].clone()
    lens, slots, st = run_append(y)
    assert st == mars.ST_OVERFLOW and lens.tolist() == [32, -1]
    assert (slots[22:40] == -1).all() and (slots[40:60] == -1).all()
    mine = x["table"][0].long()
    others = [i for i in range(before.shape[0]) if i not in mine.tolist()]
    assert torch.equal(before[others], y["k_pool"][others])


# -------------------------------------------------------------------- used together

def prefill(x, parts, hq, hkv, d):
    """A batch of prompts put into the cache in parts: attention of each part over what is
    cached, then the append, lengths kept on the device."""
    lens, n = x["lens"], x["n"]
    y = cuda(x)
    cur, new = torch.zeros(len(lens), dtype=torch.int32, device="cuda"), None
    out = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = x["cu"].tolist()
    for part in range(parts):
        cuts = [(m * part // parts, m * (part + 1) // parts) for m in lens]
        rows = torch.cat([torch.arange(starts[s] + a, starts[s] + b) for s, (a, b) in enumerate(cuts)]).cuda()
        cu = torch.tensor(np.cumsum([0] + [b - a for a, b in cuts]), dtype=torch.int32, device="cuda")
        q, k, v = (y[c][rows].contiguous() for c in "qkv")
        o = torch.empty(len(rows), hq, d, dtype=torch.bfloat16, device="cuda")
        ws = workspace(packed.OP_ATTN_CHUNK, len(lens), len(rows), hq, hkv, d, max(lens))
        packed.mars_attn_chunk(q, k, v, cu, y["k_pool"], y["v_pool"], y["table"], cur, max(lens), o,
                             ws, status=st)
        new = torch.empty_like(cur)
        packed.mars_kv_append(k, v, cu, cur, y["table"], y["k_pool"], y["v_pool"], new_lens=new, status=st)
        cur, out[rows] = new, o
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and cur.tolist() == lens
    return y, out, cur


@pytest.mark.parametrize("heads", [(4, 2, 64), (14, 2, 64), (7, 1, 128)], ids=str)
def test_prefill_in_parts_then_decode(heads):
    """A prompt's chunks, the append, then the framework's decode attention over the cache."""
    hq, hkv, d = heads
    lens, B = [150, 33, 260], 4
    x = make(lens, hq, hkv, d, seed=11, old=[0, 0, 0], spare_pages=6)
    y, out, cur = prefill(x, 3, hq, hkv, d)
    o, lse, _ = run_packed(y, fill=0.0)
    check_packed(x, out, lse, fill=0.0)        # the parts give the whole prompt's rows
    g = torch.Generator().manual_seed(1)
    q, kb, vb = (torch.randn(3, B, h, d, generator=g).to(torch.bfloat16) for h in (hq, hkv, hkv))
    od = torch.empty(3, B, hq, d, dtype=torch.float32, device="cuda")
    ws = torch.empty(mars.mars_workspace_bytes(mars.OP_DECODE_ATTN, 3, B, hq, hkv, d, max_len=260) + 16,
                     dtype=torch.uint8, device="cuda")
    # the decode kernel multiplies the free slots of the last page by weights of 0
    mars.mars_decode_attn(q.cuda(), kb.cuda(), vb.cuda(), y["k_pool"], y["v_pool"], y["table"], cur,
                          260, od, ws)
    torch.cuda.synchronize()
    cu, f = x["cu"].tolist(), f64
    for s in range(3):
        for h in range(hq):
            u = h // (hq // hkv)
            K = np.concatenate([f(x["k"][cu[s]:cu[s + 1], u]), f(kb[s, :, u])])
            V = np.concatenate([f(x["v"][cu[s]:cu[s + 1], u]), f(vb[s, :, u])])
            assert np.abs(causal_weights(f(q[s, :, h]), K) @ V - f(od[s, :, h])).max() <= 1e-2


def test_calls_in_a_graph_and_on_another_stream():
    x = make([40, 200], 14, 2, 64, seed=12, old=[2100, 300])
    y = cuda(x)
    want, _ = run_chunk(y, hint=2400)
    want_p, want_lse, _ = run_packed(y)
    n, hq, d = y["q"].shape
    o, op = torch.zeros_like(want), torch.zeros_like(want_p)
    lse = torch.zeros_like(want_lse)
    ws = workspace(packed.OP_ATTN_CHUNK, 2, n, hq, 2, d, 2400)
    wp = workspace(packed.OP_ATTN_PACKED, 2, n, hq, 2, d)

    def step(stream=None):
        packed.mars_attn_chunk(y["q"], y["k"], y["v"], y["cu"], y["k_pool"], y["v_pool"], y["table"],
                             y["old"], 2400, o, ws, stream=stream)
        packed.mars_attn_packed(y["q"], y["k"], y["v"], y["cu"], op, wp, lse=lse, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert same(o, want) and same(op, want_p) and same(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        o.zero_(), op.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(o, want) and same(op, want_p) and same(lse, want_lse)


def test_bindings_refuse_what_the_calls_in_c_decline():
    """The same errors whether the call goes through C first (current stream) or not."""
    x = make([20, 3], 4, 2, 64, seed=40, old=[30, 5])
    y = cuda(x)
    n = y["n"]
    o, ws = torch.zeros_like(y["do"]), torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    base = dict(q=y["q"], k=y["k"], v=y["v"], cu_seqlens=y["cu"], k_pool=y["k_pool"],
                v_pool=y["v_pool"], block_table=y["table"], seq_lens=y["old"], max_len_hint=50, o=o,
                workspace=ws)
    packed.mars_attn_chunk(**base)
    want = o.clone()
    # an integer scale is declined in C and taken here
    packed.mars_attn_chunk(**base, scale=0)
    assert same(o, want)
    bad = [("q", y["q"].float(), TypeError), ("k", y["k"][:-1], ValueError), ("v", None, TypeError),
           ("o", o.cpu(), ValueError), ("o", o.transpose(0, 1), ValueError),
           ("cu_seqlens", y["cu"].long(), TypeError), ("seq_lens", y["old"][:1], ValueError),
           ("block_table", y["table"][0], ValueError), ("k_pool", y["k_pool"][:, :1], ValueError),
           ("workspace", ws.float(), TypeError), ("max_len_hint", 1 << 31, ValueError),
           ("max_len_hint", -1, mars.MarsError), ("workspace", ws[:0], mars.MarsError)]
    side = torch.cuda.current_stream()
    for name, value, error in bad:
        hint = {"max_len_hint": 100000} if name == "workspace" else {}
        for stream in (None, side):
            with pytest.raises(error):
                packed.mars_attn_chunk(**{**base, **hint, name: value}, stream=stream)
    torch.cuda.synchronize()
    assert same(o, want) and n == len(o)


# ------------------------------------------------------------------- ends of the ranges

# few rows (packed_rows_kernel), and many (pair_kernel)
HINTED = [([3, 1], [2000, 1300], (14, 2, 64)),
          ([301, 40, 0, 217, 18, 1, 203, 37, 590], [300, 0, 77, 1000, 513, 129, 5, 2700, 16], (28, 4, 128))]


@pytest.mark.parametrize("hint", [0, 1, (1 << 31) - 127, (1 << 31) - 1])
@pytest.mark.parametrize("lens, old, heads", HINTED, ids=["few", "many"])
def test_chunk_hints_of_nothing_and_without_bound(lens, old, heads, hint):
    """Too small a hint leaves lists whole, the largest sizes the splits for lists of 2^31 keys."""
    x = make(lens, *heads, seed=41, old=old, tail=2)
    o, st = run_chunk(cuda(x), hint=hint)
    assert st == 0
    check_chunk(x, o)


def poison_page_zero(x):
    """Page 0, which is loaded in the place of a page that may not be read, is unused and holds NaN."""
    other = int(x["unused"][0])
    if other:
        x["table"][x["table"] == 0] = other
    assert not (x["table"] == 0).any()
    x["k_pool"][0] = x["v_pool"][0] = float("nan")


@pytest.mark.parametrize("lens, old, heads", HINTED, ids=["few", "many"])
def test_chunk_a_page_loaded_for_an_unmapped_one_has_no_effect(lens, old, heads):
    x = make(lens, *heads, seed=42, old=old, tail=2)
    poison_page_zero(x)
    x["table"][0, 3] = -1
    x["table"][0, 7] = x["k_pool"].shape[0]
    x["table"][1 if old[1] else 3, 0] = 1 << 20
    o, st = run_chunk(cuda(x))
    assert st == mars.ST_NOPAGE
    check_chunk(x, o)


# ------------------------------------------------- NaN, infinities, maxima that grow and fall
#
# The same on every form: lists that are whole, split (packed_rows_kernel) or divided among CTAs
# (pair_kernel). `old` None: mars_attn_packed.
FORMS = {"few-whole": ([200, 90], None, (4, 2, 64)), "few-split-packed": ([900], None, (4, 1, 64)),
         "one-token-split": ([1, 1, 1], [128, 1, 2300], (14, 2, 64)),
         "few-split": ([130, 2], [1000, 1700], (7, 1, 128)),
         "one-token-63-splits": ([1, 2], [40000, 17], (2, 1, 64)),
         "many-divided-64": ([2800], None, (14, 2, 64)),
         "many-divided": ([1400], None, (28, 4, 128)),
         "many-whole": ([(331 * i) % 500 + 40 for i in range(22)], None, (28, 4, 128)),
         "many-chunks-divided": HINTED[1],
         "many-chunks-whole": ([(331 * i) % 300 + 20 for i in range(28)],
                               [(217 * i) % 900 for i in range(28)], (28, 4, 128))}


def run_form(x):
    """(o, lse or None)"""
    y = cuda(x)
    if "old" in x:
        o, st = run_chunk(y)
        lse = None
    else:
        o, lse, st = run_packed(y)
    assert st == 0
    return o, lse


def positive(x):
    """The first coordinate of every query positive, so that an infinite key coordinate there gives
    infinite scores."""
    x["q"][..., 0] = x["q"][..., 0].abs() + 0.25


def assert_only(rows, before, after):
    """NaN in these rows, all others bit-equal to the run before."""
    (o, lse), (o2, lse2) = before, after
    hit = torch.zeros(len(o), dtype=torch.bool)
    hit[rows] = True
    assert o2.cpu()[hit].isnan().all() and same(o[~hit.to(o.device)], o2[~hit.to(o.device)])
    if lse is not None:
        assert lse2.cpu()[:, hit].isnan().all()
        assert same(lse[:, ~hit.to(o.device)], lse2[:, ~hit.to(o.device)])


@pytest.mark.parametrize("form", FORMS)
def test_a_query_of_nan_gives_nan(form):
    lens, old, heads = FORMS[form]
    x = make(lens, *heads, seed=43, old=old, tail=1)
    before = run_form(x)
    row = int(x["cu"][1]) - 1
    x["q"][row] = float("nan")
    assert_only([row], before, run_form(x))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("form", FORMS)
def test_a_score_of_nan_or_infinity_gives_nan(form, value):
    """One of the sequence's own keys: the rows from it on; a cached one: all of them."""
    lens, old, heads = FORMS[form]
    x = make(lens, *heads, seed=44, old=old, tail=1)
    positive(x)
    before = run_form(x)
    s = max(range(len(lens)), key=lambda i: lens[i])
    a, b = int(x["cu"][s]), int(x["cu"][s + 1])
    key = (a + b) // 2
    keep = x["k"][key, :, 0].clone()
    x["k"][key, :, 0] = value
    assert_only(list(range(key, b)), before, run_form(x))
    if old is not None and old[s] > 70:
        x["k"][key, :, 0] = keep
        x["k_pool"][x["table"][s, 70 // PAGE], :, 70 % PAGE, 0] = value
        assert_only(list(range(a, b)), before, run_form(x))


def slope(x, profile, top=100.0):
    """Scores that rise by `top` along the keys, fall by it, or rise and fall again (in natural
    units, on top of the normal ones)."""
    d = x["q"].shape[2]
    x["q"][..., 0] = 4.0
    unit = top * np.sqrt(d) / 4.0
    for s, m in enumerate(x["lens"]):
        p = int(x["old"][s]) if "old" in x else 0
        at = np.arange(p + m) / max(p + m - 1, 1)
        z = {"rising": at, "falling": 1.0 - at, "bump": 1.0 - np.abs(2.0 * at - 1.0)}[profile]
        z = torch.tensor(unit * z).to(torch.bfloat16)
        a = int(x["cu"][s])
        x["k"][a:a + m, :, 0] = z[p:, None]
        for t in range(p):
            x["k_pool"][x["table"][s, t // PAGE], :, t % PAGE, 0] = z[t]


@pytest.mark.parametrize("profile", ["rising", "falling", "bump"])
@pytest.mark.parametrize("form", FORMS)
def test_maxima_that_grow_and_fall_along_the_keys(form, profile):
    """Rows whose maximum grows by far more than the 2^8 from which O is rescaled, and parts of a
    list with very different maxima.

    A score is a sum of d products in 32 bits, exact before the sum: with |z| its scaled absolute
    sum, z is off by at most E = (d / 16 + 16) 2^-23 |z| (a step of 16 products each, up to 16
    roundings inside a step, each of at most a unit in the last place). Weights then change by
    factors within 1 +- E before and after they are normalised: a row of O by at most 2 E max|v|,
    the log2 statistic by log2(e) E."""
    lens, old, heads = FORMS[form]
    x = make(lens, *heads, seed=45, old=old, tail=1)
    slope(x, profile)
    o, lse = run_form(x)
    o, cu, (hq, hkv, d) = f64(o), x["cu"].tolist(), heads
    step = (d / 16 + 16) * 2.0 ** -23
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        p = old[s] if old is not None else 0
        at = [(int(x["table"][s, t // PAGE]), t % PAGE) for t in range(p)]
        for h in range(hq if b > a else 0):
            u = h // (hq // hkv)
            K, V = f64(x["k"][a:b, u]), f64(x["v"][a:b, u])
            if p:
                pages, slots = (torch.tensor(c) for c in zip(*at))
                K = np.concatenate([f64(x["k_pool"][pages, u, slots]), K])
                V = np.concatenate([f64(x["v_pool"][pages, u, slots]), V])
            q = f64(x["q"][a:b, h])
            P = causal_weights(q, K)
            E = step * (np.abs(q) @ np.abs(K).T).max() / np.sqrt(d)
            ref = P @ V
            assert_within_bound(o[a:b, h], ref, output_bound(P, V, ref) + 2 * E * np.abs(V).max(),
                                f"seq {s} head {h}")
            if lse is not None:
                z = np.where(np.tri(b - a, dtype=bool), q @ K.T / np.sqrt(d), -np.inf)
                m = z.max(axis=1)
                want = (m + np.log(np.exp(z - m[:, None]).sum(axis=1))) / np.log(2.0)
                err = np.abs(f64(lse[h, a:b]) - want).max()
                assert err <= LSE_TOL + 1.4426950408889634 * E + 256 * 2.0 ** -24, (s, h)


@pytest.mark.parametrize("which", ["q", "do"])
@pytest.mark.parametrize("row", [0, 77, 299])
@pytest.mark.parametrize("lens, heads", [([300, 40], (4, 2, 64)), ([300, 1200], (14, 2, 128))], ids=str)
def test_gradient_of_a_nan_row_is_nan(lens, heads, row, which):
    """dq of the row, dk and dv of the keys that it sees; dq of the others and the other sequence
    stay as they were (dk and dv of the rows behind it may be NaN)."""
    x = make(lens, *heads, seed=46, tail=2)
    got = []
    for bad in (False, True):
        if bad:
            x[which][row] = float("nan")
        y = cuda(x)
        o, lse, _ = run_packed(y)
        got.append(run_grad(y, o, lse, y["do"]))
        assert got[-1][3] == 0
    (dq, dk, dv, _), (dq2, dk2, dv2, _) = got
    assert dq2[row].isnan().all() and dk2[:row + 1].isnan().all() and dv2[:row + 1].isnan().all()
    others = [i for i in range(x["n"]) if i != row]
    assert same(dq[others], dq2[others])
    assert same(dk[lens[0]:], dk2[lens[0]:]) and same(dv[lens[0]:], dv2[lens[0]:])


@pytest.mark.parametrize("what", ["table", "pool", "both"])
def test_append_to_an_empty_pool_or_table(what):
    """Nothing can be written: the lengths stay, no row has a slot, and the status says why."""
    x = make([20, 0, 3], 4, 2, 64, seed=47, old=[5, 7, 16])
    y = cuda(x)
    if what != "pool":
        y["table"] = y["table"][:, :0].contiguous()
    if what != "table":
        y["k_pool"], y["v_pool"] = y["k_pool"][:0], y["v_pool"][:0]
    before = y["k_pool"].clone(), y["v_pool"].clone()
    for stream in (None, torch.cuda.current_stream()):
        lens, slots, st = run_append(y, stream=stream)
        assert st == (mars.ST_NOPAGE if what == "pool" else mars.ST_OVERFLOW)
        assert lens.tolist() == [5, 7, 16] and (slots == -1).all()
    assert same(before[0], y["k_pool"]) and same(before[1], y["v_pool"])


# ------------------------------------------------- groups, offsets, a replayed serving loop

@pytest.mark.parametrize("lens, heads", [([300, 77, 1], (96, 1, 64)), ([377, 40], (130, 1, 64)),
                                         ([500, 3, 130], (33, 1, 128)), ([700, 260, 5], (40, 40, 64)),
                                         ([301, 90], (128, 1, 128))], ids=str)
def test_packed_many_rows_of_other_groups(lens, heads):
    """pair_kernel with row tiles of one token, of 128 and in between, and its gradient."""
    x = make(lens, *heads, seed=48, tail=1)
    y = cuda(x)
    o, lse, st = run_packed(y)
    assert st == 0
    check_packed(x, o, lse)
    dq, dk, dv, st = run_grad(y, o, lse, y["do"])
    assert st == 0
    check_grad(x, dq, dk, dv)
    z = make(lens, *heads, seed=49, tail=1, old=[70 * i + 200 for i in range(len(lens))])
    o, st = run_chunk(cuda(z))
    assert st == 0
    check_chunk(z, o)


def part_of(x, names, rows, **more):
    """The rows of a sequence on the CPU as a batch of their own."""
    y = {c: x[c][rows].cpu() for c in names}
    n = len(y["q"])
    return {**y, "n": n, "cu": torch.tensor([0, n], dtype=torch.int32), **more}


def test_rows_whose_offsets_pass_32_bits():
    """q, o, d_o and dq of more than 2^31 elements; the first sequence and the last."""
    hq, hkv, d, m, batch = 28, 4, 128, 650, 960
    n = m * batch + 3
    assert n * hq * d > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(50)
    y = {c: torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
         for c, h in (("q", hq), ("k", hkv), ("v", hkv), ("do", hq))}
    y["cu"] = torch.arange(0, n - 2, m, dtype=torch.int32, device="cuda")
    o, lse, st = run_packed(y)
    assert st == 0 and (o[-3:] == 7.0).all()
    dq, dk, dv, st = run_grad(y, o, lse, y["do"], wide=False)
    assert st == 0 and (dq[-3:] == 7.0).all() and (dv[-3:] == 7.0).all()
    for a in (0, n - 3 - m):
        rows = slice(a, a + m)
        x = part_of(y, ("q", "k", "v", "do"), rows)
        check_packed(x, o[rows], lse[:, rows])
        check_grad(x, dq[rows], dk[rows], dv[rows])


def test_pools_whose_offsets_pass_32_bits():
    """Pools of more than 2^31 elements: an append to their last pages and a chunk over them."""
    lens, old, (hq, hkv, d) = [40, 3], [100, 33], (28, 4, 128)
    x = make(lens, hq, hkv, d, seed=51, old=old)
    pages = (1 << 31) // (hkv * PAGE * d) + 64
    small, shift = x["k_pool"].shape[0], pages - x["k_pool"].shape[0]
    y = cuda(x)
    y["table"] = torch.where(y["table"] >= 0, y["table"] + shift, y["table"])
    for c in ("k_pool", "v_pool"):
        big = torch.empty(pages, hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
        assert big.numel() > 1 << 31
        big[shift:] = y[c]
        y[c] = big
    o, st = run_chunk(y)
    assert st == 0
    check_chunk(x, o)
    new_lens, slots, st = run_append(y)
    kp, vp, want_lens, want_slots = oracle.kv_append(
        f64(x["k"]), f64(x["v"]), x["cu"].numpy(), x["old"].numpy(), x["table"].numpy(),
        f64(x["k_pool"]), f64(x["v_pool"]), PAGE)
    assert st == 0 and (new_lens.cpu().numpy() == want_lens).all()
    assert (slots.cpu().numpy() == want_slots + shift * PAGE).all() and small + shift == pages
    assert (f64(y["k_pool"][shift:]) == kp).all() and (f64(y["v_pool"][shift:]) == vp).all()


def test_a_captured_step_over_growing_caches():
    """A token per sequence and step, captured once: lengths live on the device and grow past the
    hint; every replay gives what the calls give one by one."""
    hq, hkv, d, steps, old = 14, 2, 64, 40, [250, 0, 15, 1030]
    x = make([steps] * 4, hq, hkv, d, seed=52, old=old)
    y = cuda(x)
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    ws = workspace(packed.OP_ATTN_CHUNK, 4, 4, hq, hkv, d, 1032)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(4, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    o, cur, new = torch.zeros_like(q), y["old"].clone(), torch.zeros_like(y["old"])

    def step(kp, vp):
        packed.mars_attn_chunk(q, k, v, cu, kp, vp, y["table"], cur, 1032, o, ws, status=st)
        packed.mars_kv_append(k, v, cu, cur, y["table"], kp, vp, new_lens=new, status=st)
        cur.copy_(new)

    def loop(f):
        out = []
        cur.copy_(y["old"])
        for i in range(steps):
            for t, c in ((q, "q"), (k, "k"), (v, "v")):
                t.copy_(y[c][i::steps])
            f()
            out.append(o.clone())
        torch.cuda.synchronize()
        assert cur.tolist() == [p + steps for p in old] and int(st.item()) == 0
        return torch.stack(out, 1).flatten(0, 1)          # rows of a sequence together

    eager = y["k_pool"].clone(), y["v_pool"].clone()
    want = loop(lambda: step(*eager))
    pools = y["k_pool"].clone(), y["v_pool"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*pools)
    got = loop(graph.replay)
    assert same(got, want) and same(eager[0], pools[0]) and same(eager[1], pools[1])
    check_chunk(x, want)                                   # the same rows as one chunk


@pytest.mark.parametrize("what", ["table", "pool"])
@pytest.mark.parametrize("lens, old, heads", HINTED, ids=["few", "many"])
def test_chunk_over_lengths_without_any_page(lens, old, heads, what):
    """An empty pool, or a table without a column: the chunk's own keys are what is left."""
    x = make(lens, *heads, seed=53, old=old, tail=2)
    y = cuda(x)
    if what == "table":
        y["table"] = y["table"][:, :0].contiguous()
    else:
        y["k_pool"], y["v_pool"] = y["k_pool"][:0], y["v_pool"][:0]
    o, st = run_chunk(y)
    assert st == (mars.ST_OVERFLOW if what == "table" else mars.ST_NOPAGE)
    x["old"].zero_()
    check_chunk(x, o)
