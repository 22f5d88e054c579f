"""Rotary positions, the append to the 8-bit paged cache and attention over it against the fp64
oracle (needs a GB300). Bounds are elementwise; codes, scales and slots are exact."""
import numpy as np
import pytest
import torch

import oracle
from block_masked_token_gb300 import mars, packed
from packed_util import PAGE, causal_weights, cuda, f64, make, output_bound, workspace
from parity_util import U_BF16, assert_within_bound

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (7, 1, 128), (28, 4, 128), (14, 2, 64)]
WIDE_HEADS = [(24, 1, 64), (48, 2, 128)]            # more query heads per KV head than a tile of few rows holds


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def codes(values):
    return torch.from_numpy(values).float().to(torch.float8_e4m3fn)


def make8(lens, hq, hkv, d, old, seed=0, k_spread=0.3, v_spread=0.7, **kw):
    """packed_util.make with pools of codes and scales whose sizes differ page by page."""
    x = make(lens, hq, hkv, d, seed=seed, old=old, **kw)
    rng = np.random.default_rng(seed)
    for c, spread in (("k", k_spread), ("v", v_spread)):
        y = f64(x[c + "_pool"]) * np.exp(spread * rng.normal(size=(*x[c + "_pool"].shape[:2], 1, 1)))
        s = np.array([[oracle.q8_scale(h) for h in page] for page in y], dtype=np.uint8).reshape(y.shape[:2])
        x[c + "_pool"] = codes(oracle.e4m3(y * np.exp2(127.0 - s)[..., None, None]))
        x[c + "_scale"] = torch.from_numpy(s)
    return x


def values(x, c):
    return oracle.q8_values(f64(x[c + "_pool"].float()), x[c + "_scale"].numpy())


def hint_of(x):
    return max(int(p) + m for p, m in zip(x["old"].tolist(), x["lens"]))


def run_chunk8(y, fill=7.0, hint=None, scale=0.0, ws=None, o=None, **kw):
    n, hq, d = y["q"].shape
    if o is None:
        o = torch.full((n, hq, d), fill, dtype=torch.bfloat16, device="cuda")
    st = status()
    hint = hint_of(y) if hint is None else hint
    if ws is None:
        ws = workspace(packed.OP_ATTN_CHUNK_Q8, len(y["cu"]) - 1, n, hq, y["k"].shape[1], d, hint)
    packed.mars_attn_chunk_q8(y["q"], y["k"], y["v"], y["cu"], y["k_pool"], y["v_pool"],
                              y["k_scale"], y["v_scale"], y["table"], y["old"], hint, o, ws,
                              status=st, scale=scale, **kw)
    torch.cuda.synchronize()
    return o, int(st.item())


def check_chunk8(x, o, fill=7.0, scale=None, rows=None, slack=0.0):
    """Against the definition over the pages' values; a page that is unmapped has no keys."""
    kv, vv = values(x, "k"), values(x, "v")
    o, cu, g = f64(o), x["cu"].tolist(), x["q"].shape[1] // x["k"].shape[1]
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        P = min(max(0, int(x["old"][s])), PAGE * x["table"].shape[1])
        ids = [(int(x["table"][s, p // PAGE]), p % PAGE) for p in range(P)]
        ids = [(e, c) for e, c in ids if 0 <= e < len(kv)]
        e, c = np.array([i[0] for i in ids], dtype=int), np.array([i[1] for i in ids], dtype=int)
        for u in range(x["k"].shape[1] if b > a else 0):
            K = np.concatenate([kv[e, u, c].reshape(-1, kv.shape[3]), f64(x["k"][a:b, u])])
            V = np.concatenate([vv[e, u, c].reshape(-1, kv.shape[3]), f64(x["v"][a:b, u])])
            for h in range(u * g, u * g + g):
                r = np.arange(b - a) if rows is None else np.array([i for i in rows if i < b - a], dtype=int)
                P_ = causal_weights(f64(x["q"][a:b, h]), K, scale)[r]
                ref = P_ @ V
                assert_within_bound(o[a:b, h][r], ref, output_bound(P_, V, ref) + slack,
                                    f"sequence {s} head {h}")
    outside = np.ones(x["n"], dtype=bool)
    outside[cu[0]:cu[-1]] = False
    assert (o[outside] == fill).all()


def same(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.cpu().view(torch.uint8))


CHUNKS = [([1], [0]), ([1], [1]), ([1], [50]), ([1, 1, 1], [15, 16, 17]), ([0, 3, 0, 1], [9, 127, 5, 128]),
          ([8, 8], [129, 1000]), ([18, 19, 37], [3, 700, 255]), ([150, 1], [0, 300]), ([300], [40])]


@pytest.mark.parametrize("heads", HEADS + WIDE_HEADS, ids=str)
@pytest.mark.parametrize("lens, old", CHUNKS, ids=str)
def test_chunk_matches_the_definition(lens, old, heads):
    x = make8(lens, *heads, old, seed=len(lens), tail=3, lead=1, fused=heads[0] != 4)
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check_chunk8(x, o)
    again, _ = run_chunk8(cuda(x))
    assert same(o, again)


MANY = [([1] * 40, [(131 * i) % 900 for i in range(40)], (28, 4, 128)),
        ([16] * 20, [(517 * i) % 2000 for i in range(20)], (28, 4, 128)),
        ([1], [20000], (7, 1, 128)), ([2, 1], [9000, 30], (14, 2, 64)),
        ([(i * 11) % 5 for i in range(300)], [(i * 37) % 60 for i in range(300)], (4, 2, 64)),
        ([700, 1, 3, 260, 18, 19], [500, 1500, 0, 33, 900, 64], (28, 4, 128)),
        ([900, 5, 1], [100, 4000, 7], (16, 16, 128)), ([1500], [2000], (14, 2, 64)),
        ([3, 2], [200, 90], (130, 1, 64)), ([2, 5], [300, 129], (96, 1, 64))]


@pytest.mark.parametrize("lens, old, heads", MANY, ids=lambda v: str(v)[:24])
def test_chunk_of_many_items(lens, old, heads):
    x = make8(lens, *heads, old, seed=41, tail=2)
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check_chunk8(x, o, rows=[0, 1, 7, 17, 18, 127, 128, 255, 256, 699, 899, 1499])
    again, _ = run_chunk8(cuda(x))
    assert same(o, again)


@pytest.mark.parametrize("hint", [0, 1, 100, 900, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("lens, old, heads", [([1, 4], [800, 60], (28, 4, 128)),
                                              ([3, 4], [800, 60], (24, 1, 128)),
                                              ([700, 1, 800], [500, 900, 20], (28, 4, 128))],
                         ids=["few", "middle", "many"])
def test_chunk_hint_is_no_bound(lens, old, heads, hint):
    x = make8(lens, *heads, old, seed=42)
    o, st = run_chunk8(cuda(x), hint=hint)
    assert st == 0
    check_chunk8(x, o, rows=[0, 3, 300, 699, 799])


@pytest.mark.parametrize("lens, old, heads", [([2, 20], [400, 90], (7, 1, 128)),
                                              ([2, 20], [400, 90], (24, 1, 128)),
                                              ([900, 700], [400, 90], (28, 4, 128))], ids=["few", "middle", "many"])
def test_chunk_unmapped_pages_and_cut_lengths(lens, old, heads):
    x = make8(lens, *heads, old, seed=43)
    x["table"][0, 3], x["table"][0, 24], x["table"][1, :] = -1, 1 << 20, -7
    o, st = run_chunk8(cuda(x))
    assert st == mars.ST_NOPAGE
    check_chunk8(x, o, rows=[0, 1, 19, 500, 899])
    x["old"] = torch.tensor([-3, 1 << 30], dtype=torch.int32)
    o, st = run_chunk8(cuda(x), hint=1600)
    assert st & mars.ST_OVERFLOW
    check_chunk8(x, o, rows=[0, 1, 19, 500, 899])
    x["cu"][1] = -4
    o, st = run_chunk8(cuda(x), hint=1600)
    assert st & mars.ST_BADSEQ
    x["cu"][1] = 0
    check_chunk8(x, o, rows=[0, 1, 500])


@pytest.mark.parametrize("lens, heads", [([3], (7, 1, 128)), ([3], (24, 1, 128)), ([1400], (28, 4, 128))], ids=["few", "middle", "many"])
def test_chunk_empty_pool(lens, heads):
    x = make8(lens, *heads, [0], seed=44)
    for c in ("k", "v"):
        x[c + "_pool"], x[c + "_scale"] = x[c + "_pool"][:0], x[c + "_scale"][:0]
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check_chunk8(x, o, rows=[0, 2, 700, 1399])
    x["old"] = torch.tensor([40], dtype=torch.int32)
    x["table"] = torch.zeros(1, 3, dtype=torch.int32)
    o, st = run_chunk8(cuda(x))
    assert st == mars.ST_NOPAGE
    check_chunk8(x, o, rows=[0, 2, 700, 1399])


@pytest.mark.parametrize("lens, old, heads", [([3, 1], [200, 37], (14, 2, 64)),
                                              ([3, 20], [200, 37], (24, 1, 128)),
                                              ([1400, 1], [200, 37], (28, 4, 128))], ids=["few", "middle", "many"])
def test_chunk_what_no_row_may_read_has_no_effect(lens, old, heads):
    """NaN codes in free slots and unused pages, scales of pages that hold nothing, other rows."""
    x = make8(lens, *heads, old, seed=45, tail=9, spare_pages=3)
    o, st = run_chunk8(cuda(x))
    for c in ("k", "v"):
        raw = x[c + "_pool"].view(torch.uint8)
        for s, P in enumerate(old):
            raw[x["table"][s, P // PAGE], :, P % PAGE:] = 0x7f
            for lp in range(P // PAGE + 1, -(-(P + lens[s]) // PAGE)):
                raw[x["table"][s, lp]] = 0xff
                x[c + "_scale"][x["table"][s, lp]] = 255
        raw[x["unused"].long()] = 0x7f
    x["qkv"][sum(lens):] = float("nan")
    o2, st2 = run_chunk8(cuda(x))
    assert st == st2 == 0
    assert same(o[:sum(lens)], o2[:sum(lens)])


@pytest.mark.parametrize("lens, heads", [([3], (7, 1, 128)), ([3], (24, 1, 128)), ([1400], (28, 4, 128))], ids=["few", "middle", "many"])
def test_chunk_nan_codes_are_not_lost(lens, heads):
    x = make8(lens, *heads, [300], seed=46)
    for c in ("k", "v"):
        y = dict(x)
        y[c + "_pool"] = x[c + "_pool"].clone()
        y[c + "_pool"].view(torch.uint8)[x["table"][0, 5], :, 3, 11] = 0x7f
        o, st = run_chunk8(cuda(y))
        assert st == 0
        assert torch.isnan(o).all() if c == "k" else torch.isnan(o[:, :, 11]).all()
    q = make8(lens, *heads, [300], seed=46)
    q["q"][1, 2] = float("nan")
    o, st = run_chunk8(cuda(q))
    assert st == 0 and torch.isnan(o[1, 2]).all()
    o[1, 2] = 0
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("profile", ["rising", "falling", "peak"])
@pytest.mark.parametrize("lens, heads", [([2], (7, 1, 128)), ([2], (24, 1, 128)), ([1300], (28, 4, 128))], ids=["few", "middle", "many"])
def test_chunk_maxima_that_grow_and_fall(lens, heads, profile):
    """Scores that grow by far more than the lazy rescaling lets pass, page by page."""
    x = make8(lens, *heads, [1000], seed=47, k_spread=0.0)
    step = {"rising": np.arange(63) // 8, "falling": 7 - np.arange(63) // 8,
            "peak": 7 - np.abs(np.arange(63) - 31) // 5}[profile]
    for lp in range(63):
        x["k_scale"][x["table"][0, lp]] = int(x["k_scale"].min()) + int(step[lp]) - 4
    o, st = run_chunk8(cuda(x))
    assert st == 0
    # scores of up to some hundreds: 2^4 those of the model's inputs, and so is the upstream error
    # of a weight, 2^-14; the absolute errors of the weights sum to 2 * 16 * 2^-14 at most
    slack = 2 * 16 * 2.0 ** -14 * np.abs(values(x, "v")).max()
    check_chunk8(x, o, rows=[0, 1, 600, 1299], slack=slack)


@pytest.mark.parametrize("lens, heads", [([2], (7, 1, 128)), ([2], (24, 1, 128)), ([1300], (28, 4, 128))], ids=["few", "middle", "many"])
def test_chunk_scales_far_apart(lens, heads):
    """V scales over the whole range page by page (the tiny ones first, last and in between), a
    zero page, and new V rows of another size than the cache's."""
    x = make8(lens, *heads, [900], seed=48)
    for exps, own in ((list(range(-40, 0, 7)), 1.0), ([40, -40, 0], 1.0), ([-40, -30], 2.0 ** -30),
                      ([30, 40], 2.0 ** 20)):
        for lp in range(57):
            x["v_scale"][x["table"][0, lp]] = 127 + exps[lp % len(exps)]
        x["v_pool"].view(torch.uint8)[x["table"][0, 4]] = 0
        y = dict(x, v=(x["v"].float() * own).to(torch.bfloat16), fused=False)
        y["q"], y["k"] = x["q"].contiguous(), x["k"].contiguous()
        o, st = run_chunk8(cuda(y))
        assert st == 0
        check_chunk8(y, o, rows=[0, 1, 600, 1299])

# Rows (token, head) of a KV head around what one tile of the few-row kernel holds, 8 and 16, and four
# such tiles; sequences of many rows among empty ones.
FEW = [([1] * 5, (8, 1, 128)), ([2, 1, 2], (8, 2, 64)), ([3, 1], (12, 3, 128)), ([4] * 3, (16, 4, 64)),
       ([5] * 3, (16, 4, 128)), ([8, 0, 8], (1, 1, 128)), ([9, 8], (1, 1, 64)), ([16, 16], (2, 2, 128)),
       ([17, 16], (1, 1, 128)), ([1] * 4, (16, 1, 128)), ([1] * 3, (9, 1, 64)), ([2] * 3, (9, 1, 128)),
       ([8, 8], (28, 4, 128)), ([16], (14, 2, 64)), ([64], (1, 1, 128)), ([65], (1, 1, 64)),
       ([64], (28, 4, 128)), ([40, 3], (14, 2, 64)),
       ([300] + [0] * 39, (2, 2, 128)), ([0] * 30 + [140, 0, 0, 1], (4, 4, 64)), ([150] + [0] * 80, (14, 2, 64))]


@pytest.mark.parametrize("lens, heads", FEW, ids=lambda v: str(v)[:30])
def test_chunk_of_few_rows(lens, heads):
    old = [(211 * i + 17) % 700 for i in range(len(lens))]
    x = make8(lens, *heads, old, seed=len(lens) + heads[0], tail=1)
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check_chunk8(x, o)
    again, _ = run_chunk8(cuda(x))
    assert same(o, again)


@pytest.mark.parametrize("lens, old, heads", [([1] * 2500, [(i * 7) % 40 for i in range(2500)], (4, 4, 64)),
                                              ([1], [33000], (14, 2, 64)), ([2, 1], [40001, 16], (8, 1, 128)),
                                              ([1] * 3, [9000, 0, 12345], (7, 1, 128))], ids=lambda v: str(v)[:24])
def test_chunk_of_few_rows_in_many_parts(lens, old, heads):
    """More items than a CTA lists at a time, and items that many CTAs share."""
    x = make8(lens, *heads, old, seed=6)
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check_chunk8(x, o)
    again, _ = run_chunk8(cuda(x))
    assert same(o, again)


def test_chunk_of_a_page_mapped_twice():
    x = make8([1, 2], 8, 2, 64, [90, 200], seed=7)
    x["table"][0, 3] = x["table"][0, 1]
    x["table"][1, :4] = x["table"][0, :4]
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check_chunk8(x, o)


@pytest.mark.parametrize("heads", [(7, 1, 128), (14, 2, 64)], ids=str)
def test_chunk_calls_in_a_row_share_a_workspace(heads):
    """Calls whose kernels start early, each over its own data, without a wait between them."""
    sets = [make8(lens, *heads, old, seed=50 + i) for i, (lens, old) in enumerate(
        [([1, 1], [5000, 3000]), ([2, 1], [100, 6000]), ([1, 9], [900, 1]), ([30, 1], [700, 2500]), ([1], [7777])])]
    on = [cuda(x) for x in sets]
    size = max(packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, len(y["cu"]) - 1, y["q"].shape[0], *heads,
                                                  hint_of(y)) for y in on)
    ws = torch.full((size,), 0xa5, dtype=torch.uint8, device="cuda")
    outs = [[torch.full_like(y["q"].contiguous(), 7.0) for y in on] for _ in range(6)]
    st = status()
    hints = [hint_of(y) for y in on]
    for o in outs:
        for y, out, hint in zip(on, o, hints):
            packed.mars_attn_chunk_q8(y["q"], y["k"], y["v"], y["cu"], y["k_pool"], y["v_pool"], y["k_scale"],
                                      y["v_scale"], y["table"], y["old"], hint, out, ws, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, out in zip(sets, outs[0]):
        check_chunk8(x, out)
    for o in outs[1:]:
        assert all(same(a, b) for a, b in zip(o, outs[0]))


def test_chunk_replayed_with_other_lengths():
    """A captured call is replayed while the cached lengths change: the parts are cut elsewhere."""
    x = make8([1, 1, 1], 7, 1, 128, [6000, 2000, 400], seed=8)
    y = cuda(x)
    ws = workspace(packed.OP_ATTN_CHUNK_Q8, 3, y["q"].shape[0], 7, 1, 128, 6001)
    o = torch.full_like(y["q"].contiguous(), 7.0)
    run_chunk8(y, hint=6001, ws=ws, o=o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        packed.mars_attn_chunk_q8(y["q"], y["k"], y["v"], y["cu"], y["k_pool"], y["v_pool"], y["k_scale"], y["v_scale"],
                                  y["table"], y["old"], 6001, o, ws)
    for old in ([6000, 2000, 400], [10, 1999, 0], [5999, 0, 17], [6000, 2000, 400]):
        y["old"].copy_(torch.tensor(old, dtype=torch.int32))
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check_chunk8({**x, "old": torch.tensor(old, dtype=torch.int32)}, o)


def test_chunk_scale_argument_and_other_stream():
    x = make8([3, 1], 14, 2, 64, [150, 600], seed=49)
    y = cuda(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, st = run_chunk8(y, scale=0.3, stream=s)
    assert st == 0
    slack = 4 * 2.0 ** -14 * np.abs(values(x, "v")).max()       # scores 2.4 times the model's
    check_chunk8(x, o, scale=0.3, slack=slack)
    with torch.cuda.stream(s):
        o2, _ = run_chunk8(y, scale=0.3)
    assert same(o, o2)


def test_chunk_calls_at_once_on_two_streams():
    xs = [make8([16] * 9, 28, 4, 128, [700] * 9, seed=50), make8([1] * 30, 28, 4, 128, [1500] * 30, seed=51)]
    ys = [cuda(x) for x in xs]
    alone = [run_chunk8(y)[0] for y in ys]
    streams = [torch.cuda.Stream() for _ in ys]
    outs = [torch.zeros_like(a) for a in alone]
    ws = [workspace(packed.OP_ATTN_CHUNK_Q8, len(y["cu"]) - 1, y["n"], 28, 4, 128, hint_of(y)) for y in ys]
    torch.cuda.synchronize()
    for _ in range(10):
        for y, s, o, w in zip(ys, streams, outs, ws):
            packed.mars_attn_chunk_q8(y["q"], y["k"], y["v"], y["cu"], y["k_pool"], y["v_pool"], y["k_scale"],
                                      y["v_scale"], y["table"], y["old"], hint_of(y), o, w, stream=s)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(alone, outs))


# ------------------------------------------------------------------------------- append


def run_append8(y, counts=None, **kw):
    lens = torch.full((len(y["lens"]),), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((y["n"],), -9, dtype=torch.int32, device="cuda")
    st = status()
    packed.mars_kv_append_q8(y["k"], y["v"], y["cu"], y["old"], y["table"], y["k_pool"], y["v_pool"],
                             y["k_scale"], y["v_scale"], counts=counts, new_lens=lens, slots=slots, status=st, **kw)
    torch.cuda.synchronize()
    return lens, slots, int(st.item())


def check_append8(x, y, lens, slots, counts=None):
    """y: x on the GPU after the append. Bytes that the append does not write stay."""
    *want, wl, ws = oracle.kv_append_q8(f64(x["k"]), f64(x["v"]), x["cu"].numpy(), x["old"].numpy(), x["table"].numpy(),
                                        f64(x["k_pool"].float()), f64(x["v_pool"].float()), x["k_scale"].numpy(),
                                        x["v_scale"].numpy(), PAGE, counts)
    np.testing.assert_array_equal(lens.cpu().numpy(), wl)
    inside = slice(int(x["cu"][0]), int(x["cu"][-1]))
    np.testing.assert_array_equal(slots.cpu().numpy()[inside], ws[inside])
    outside = np.ones(x["n"], dtype=bool)
    outside[inside] = False
    assert (slots.cpu().numpy()[outside] == -9).all()
    for c, pool, scale in (("k", want[0], want[2]), ("v", want[1], want[3])):
        np.testing.assert_array_equal(y[c + "_scale"].cpu().numpy(), scale)
        np.testing.assert_array_equal(f64(y[c + "_pool"].float()), pool)


@pytest.mark.parametrize("heads", [(2, 2, 64), (4, 4, 128), (1, 1, 128), (9, 9, 64)], ids=str)
@pytest.mark.parametrize("lens, old", CHUNKS + [([5, 16, 33], [11, 15, 31]), ([2] * 40, list(range(40)))], ids=str)
def test_append_matches_oracle(lens, old, heads):
    x = make8(lens, *heads, old, seed=len(lens), tail=3, lead=2, v_spread=2.0)
    y = cuda(x)
    lens_, slots, st = run_append8(y)
    assert st == 0
    check_append8(x, y, lens_, slots)


@pytest.mark.parametrize("counts", [[0, 5, 99, -3], [7, 0, 1, 16]])
def test_append_of_counts(counts):
    x = make8([7, 20, 18, 16], 2, 2, 128, [10, 16, 15, 31], seed=52)
    y = cuda(x)
    lens, slots, st = run_append8(y, torch.tensor(counts, dtype=torch.int32, device="cuda"))
    assert st == 0
    check_append8(x, y, lens, slots, counts)


def test_append_of_large_small_and_infinite_rows():
    x = make8([40, 6], 2, 2, 64, [5, 16], seed=53, fused=False)
    x["k"][3, 0, 5], x["k"][4, 1, 6], x["v"][20, 0, 7] = float("inf"), float("nan"), float("-inf")
    x["k"][12:28] *= 2.0 ** 60
    x["v"][12:28] *= 2.0 ** -70
    x["v"][40:46] = 0
    x["k"][40:46, 0, :8] = torch.tensor([448.0, 449, -450, 1e30, -1e38, 3e-39, -0.0, 0.0]).to(torch.bfloat16)
    y = cuda(x)
    lens, slots, st = run_append8(y)
    assert st == 0
    check_append8(x, y, lens, slots)


def test_append_past_the_table_into_holes_and_negative_lengths():
    x = make8([40, 20, 33, 5], 2, 2, 64, [10, 16, 0, 3], seed=54)
    x["table"][0, 2] = -1
    x["table"][1, 1] = 1 << 25
    x["old"][3] = -2
    y = cuda(x)
    lens, slots, st = run_append8(y)
    assert st == mars.ST_NOPAGE | mars.ST_OVERFLOW
    check_append8(x, y, lens, slots)
    x = make8([40], 2, 2, 64, [16 * 3 - 4], seed=55)
    x["table"] = x["table"][:, :4].contiguous()
    y = cuda(x)
    lens, slots, st = run_append8(y)
    assert st == mars.ST_OVERFLOW and lens.tolist() == [64]
    check_append8(x, y, lens, slots)
    x = make8([3], 2, 2, 64, [0], seed=56)
    for c in ("k", "v"):
        x[c + "_pool"], x[c + "_scale"] = x[c + "_pool"][:0], x[c + "_scale"][:0]
    y = cuda(x)
    lens, slots, st = run_append8(y)
    assert st == mars.ST_NOPAGE and lens.tolist() == [0] and slots.tolist() == [-1] * 3


def test_append_bad_boundaries_are_cut():
    x = make8([20, 20, 10], 2, 2, 64, [5, 0, 20], seed=57)
    x["cu"] = torch.tensor([0, 40, 30, 50], dtype=torch.int32)
    x["table"] = torch.arange(15, dtype=torch.int32).view(3, 5) % len(x["k_pool"])
    y = cuda(x)
    lens, slots, st = run_append8(y)
    assert st & mars.ST_BADSEQ
    x["cu"] = torch.tensor([0, 40, 40, 50], dtype=torch.int32)
    z = cuda(x)
    l2, s2, _ = run_append8(z)
    assert same(lens, l2) and same(slots, s2) and same(y["k_pool"], z["k_pool"])


# ------------------------------------------------------------------------------- rotary


def run_rotary(y, freq, seq_lens=None, in_place=False, fill=7.0, **kw):
    q, k, st = y["q"], y["k"], status()
    qo = q if in_place else torch.full(q.shape, fill, dtype=q.dtype, device="cuda")
    ko = k if in_place else torch.full(k.shape, fill, dtype=k.dtype, device="cuda")
    packed.mars_rotary(q, k, y["cu"], freq.cuda(), qo, ko, seq_lens=seq_lens, status=st, **kw)
    torch.cuda.synchronize()
    return qo, ko, int(st.item())


def check_rotary(x, got, old, freq, fill, **kw):
    cu = x["cu"].tolist()
    outside = np.ones(x["n"], dtype=bool)
    outside[cu[0]:cu[-1]] = False
    factor = abs(kw.get("factor", 1.0))
    for c, o in zip("qk", got):
        y, o = f64(x[c]), f64(o)
        ref = oracle.rotary(y, cu, old, freq.numpy(), **kw)
        # the angle, a fraction of a turn rounded to 24 bits, is off by pi 2^-24, sincospi by 2^-23
        # at most, the product with the factor and the two products and their sum by 2^-24 each of
        # values below |a| + |b|: 2^-20 in all; then the result is rounded to bf16
        half = len(freq)
        mag = np.zeros_like(y)
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if kw.get("interleaved") else (slice(0, half), slice(half, 2 * half))
        mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
        e = 2.0 ** -20 * factor * mag
        bound = e + U_BF16 * (np.abs(ref) + e)
        inside = ~outside
        assert_within_bound(o[inside], ref[inside], bound[inside] + 1e-38, c)
        assert (o[inside][..., 2 * half:] == y[inside][..., 2 * half:]).all()
        assert (o[outside] == (f64(fill[c])[outside] if isinstance(fill, dict) else fill)).all()


@pytest.mark.parametrize("kw", [{}, {"interleaved": True}, {"inverse": True, "factor": 1.2},
                                {"interleaved": True, "inverse": True, "factor": -0.5}], ids=str)
@pytest.mark.parametrize("lens, old", [([1], [0]), ([0, 1, 0, 9], [3, 100, 2, 70000]), ([17, 8, 300], [5, 0, 131000]),
                                       ([2] * 70, list(range(70)))], ids=lambda v: str(v)[:16])
@pytest.mark.parametrize("heads, rot", [((4, 2, 64), 64), ((28, 4, 128), 128), ((7, 1, 128), 64), ((3, 3, 64), 16),
                                        ((5, 1, 128), 48), ((2, 1, 128), 112)], ids=str)
def test_rotary_matches_oracle(lens, old, heads, rot, kw):
    x = make(lens, *heads, seed=len(lens), tail=2, lead=1, fused=heads[0] != 4)
    freq, _ = packed.rotary_frequencies(rot)
    old32 = torch.tensor(old, dtype=torch.int32, device="cuda")
    y = cuda(x)
    *got, st = run_rotary(y, freq, old32, **kw)
    assert st == 0
    check_rotary(x, got, old, freq, 7.0, **kw)
    # in place: the same, and the rows of no sequence (and V beside them) are left as they were
    before = y["qkv"].clone() if x["fused"] else None
    *again, st = run_rotary(y, freq, old32, in_place=True, **kw)
    assert st == 0
    inside = slice(int(x["cu"][0]), int(x["cu"][-1]))
    assert all(same(a[inside], b[inside]) for a, b in zip(got, again))
    check_rotary(x, again, old, freq, x, **kw)
    if before is not None:
        hq, hkv = heads[:2]
        assert same(before[:, hq + hkv:], y["qkv"][:, hq + hkv:])


def test_rotary_positions_beyond_what_32_bits_resolve():
    """Angles of millions of radians, and a frequency that no base gives."""
    x = make([5, 3], 2, 2, 64, seed=60)
    old = [(1 << 24) + 1, (1 << 30) + 12345]
    freq, _ = packed.rotary_frequencies(64)
    freq[1], freq[2], freq[3] = 1.7, -0.3, 0.0
    *got, st = run_rotary(cuda(x), freq, torch.tensor(old, dtype=torch.int32, device="cuda"))
    assert st == 0
    # fp64 itself loses 2^-53 of 2^31 radians, 2^-22: within the bound's 2^-20 with the rest
    check_rotary(x, got, old, freq, 7.0)


def test_rotary_without_lengths_negative_ones_and_bad_frequencies():
    x = make([9, 4], 4, 2, 64, seed=61)
    freq, _ = packed.rotary_frequencies(32)
    *got, st = run_rotary(cuda(x), freq)
    assert st == 0
    check_rotary(x, got, [0, 0], freq, 7.0)
    *neg, st = run_rotary(cuda(x), freq, torch.tensor([-5, 0], dtype=torch.int32, device="cuda"))
    assert st == mars.ST_OVERFLOW and all(same(a, b) for a, b in zip(got, neg))
    for bad in (float("nan"), float("inf")):
        freq[3] = bad
        *nan, _ = run_rotary(cuda(x), freq)
        for a, b in zip(got, nan):
            hit = torch.zeros(64, dtype=torch.bool)
            hit[[3, 19]] = True
            assert torch.isnan(b[..., hit]).all() and same(a[..., ~hit], b[..., ~hit])
    x["cu"] = torch.tensor([0, 11, 9], dtype=torch.int32)
    *_, st = run_rotary(cuda(x), packed.rotary_frequencies(32)[0])
    assert st == mars.ST_BADSEQ


def test_rotary_gradient_undoes_the_rotation():
    """<R x, y> = <x, R' y> in fp64 over the bf16 results, up to their rounding."""
    x = make([130, 40], 28, 4, 128, seed=62)
    freq, factor = packed.rotary_frequencies(128, scaling="parts", stretch=4.0, trained=4096)
    y = cuda(x)
    up = cuda(make([130, 40], 28, 4, 128, seed=63))
    fwd, bwd = run_rotary(y, freq, factor=factor), run_rotary(up, freq, factor=factor, inverse=True)
    for a, b, u, w in zip((y["q"], y["k"]), fwd, (up["q"], up["k"]), bwd):
        a, b, u, w = f64(a), f64(b), f64(u), f64(w)
        lhs, rhs = (b * u).sum(axis=-1), (a * w).sum(axis=-1)
        room = (U_BF16 + 2.0 ** -19) * ((np.abs(b) + 1e-9) * np.abs(u) + np.abs(a) * (np.abs(w) + 1e-9)).sum(axis=-1)
        assert (np.abs(lhs - rhs) <= room).all()


# ----------------------------------------------------------------------------- together


@pytest.mark.parametrize("heads", [(28, 4, 128), (14, 2, 64)], ids=str)
def test_a_serving_step(heads):
    """Rotate, attend, append; a prompt in chunks, then decoded tokens, from one captured graph for
    the single tokens: each step against the oracle over the cache as it stands."""
    hq, hkv, d = heads
    batch, width = 3, 30
    pages = batch * width + 1
    g = torch.Generator().manual_seed(70)
    table = torch.randperm(pages, generator=g)[:batch * width].to(torch.int32).view(batch, width)
    pools = {c + "_pool": torch.full((pages, hkv, PAGE, d), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for c in "kv"}
    scales = {c + "_scale": torch.full((pages, hkv), 255, dtype=torch.uint8, device="cuda") for c in "kv"}
    freq, factor = packed.rotary_frequencies(d, scaling="linear", stretch=2.0)
    dev = dict(table=table.cuda(), freq=freq.cuda(), st=status(), **pools, **scales)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    hint = width * PAGE

    def buffers(n, per):
        cu = torch.tensor(np.cumsum([0] + per), dtype=torch.int32)
        return dict(cu=cu.cuda(), qkv=torch.zeros(n, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda"),
                    o=torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda"), new=torch.zeros_like(lens),
                    ws=workspace(packed.OP_ATTN_CHUNK_Q8, batch, n, hq, hkv, d, hint))

    def step(b):
        q, k, v = b["qkv"].split([hq, hkv, hkv], dim=1)
        packed.mars_rotary(q, k, b["cu"], dev["freq"], q, k, seq_lens=lens, factor=factor, status=dev["st"])
        packed.mars_attn_chunk_q8(q, k, v, b["cu"], dev["k_pool"], dev["v_pool"], dev["k_scale"], dev["v_scale"],
                                  dev["table"], lens, hint, b["o"], b["ws"], status=dev["st"])
        packed.mars_kv_append_q8(k, v, b["cu"], lens, dev["table"], dev["k_pool"], dev["v_pool"], dev["k_scale"],
                                 dev["v_scale"], new_lens=b["new"], status=dev["st"])
        lens.copy_(b["new"])

    def check(b, per, before, state):
        x = dict(n=sum(per), lens=per, cu=b["cu"].cpu(), old=before, table=table, **state)
        x["q"], x["k"], x["v"] = b["qkv"].cpu().split([hq, hkv, hkv], dim=1)
        check_chunk8(x, b["o"], rows=list(range(0, 200, 23)))

    def state():
        return {n: dev[n].cpu() for n in ("k_pool", "v_pool", "k_scale", "v_scale")}

    for per in ([130, 7, 16], [60, 20, 3]):
        b = buffers(sum(per), per)
        b["qkv"].copy_(torch.randn(b["qkv"].shape, generator=g))
        before, old_state = lens.cpu(), state()
        step(b)
        torch.cuda.synchronize()
        check(b, per, before, old_state)
    b = buffers(batch, [1] * batch)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(b)                                    # first calls set attributes up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for i in range(20):
        b["qkv"].copy_(torch.randn(b["qkv"].shape, generator=g))
        before, old_state = lens.cpu(), state()
        graph.replay()
        torch.cuda.synchronize()
        if i in (0, 1, 15, 19):
            check(b, [1] * batch, before, old_state)
    assert int(dev["st"].item()) == 0
    assert lens.tolist() == [190 + 21, 27 + 21, 19 + 21]


@pytest.mark.parametrize("lens, old, heads", [([1, 2], [3000, 90], (7, 1, 128)), ([20, 3], [400, 900], (28, 4, 128))],
                         ids=["few", "more"])
def test_a_captured_step_over_two_streams(lens, old, heads):
    """q is turned on one stream and k on another, each by a call that writes both; attention waits for the two.
    Every kernel starts early behind the ones before it, so that a missing wait would read what is not there yet."""
    x = make8(lens, *heads, old, seed=70)
    y = cuda(x)
    freq, _ = packed.rotary_frequencies(heads[2])
    freq, cu, n = freq.cuda(), y["cu"], y["q"].shape[0]
    hint = hint_of(y)
    ws = workspace(packed.OP_ATTN_CHUNK_Q8, len(lens), n, *heads, hint)
    bufs = [torch.zeros_like(t.contiguous()) for t in (y["q"], y["k"], y["q"], y["k"], y["q"])]
    q_in, k_in = y["q"].clone(), y["k"].clone()
    other = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            packed.mars_rotary(q_in, k_in, cu, freq, bufs[2], bufs[3], y["old"])
        packed.mars_rotary(q_in, k_in, cu, freq, bufs[0], bufs[1], y["old"])
        here.wait_stream(other)
        packed.mars_attn_chunk_q8(bufs[0], bufs[3], y["v"], cu, y["k_pool"], y["v_pool"], y["k_scale"], y["v_scale"],
                                  y["table"], y["old"], hint, bufs[4], ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = torch.Generator(device="cuda").manual_seed(5)
    for _ in range(4):
        for t in (q_in, k_in):
            t.copy_(torch.randn(t.shape, generator=rng, device="cuda"))
        for b in bufs:
            b.fill_(7.0)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        got = [b.clone() for b in bufs]
        for b in bufs:
            b.fill_(3.0)
        step()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, bufs))
        check_chunk8({**x, "q": bufs[0].cpu(), "k": bufs[3].cpu()}, got[4])


def test_rows_and_pools_whose_offsets_pass_32_bits():
    """A pool of 5.4 GB whose last pages are in use, and rows of a tensor of 4.6 GB."""
    hq, hkv, d = 8, 8, 128
    pages = (1 << 32) // (hkv * PAGE * d) + (1 << 16)
    x = make8([40, 1], hq, hkv, d, [70, 33], seed=80)
    big = {c + "_pool": torch.zeros(pages, hkv, PAGE, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for c in "kv"}
    scale = {c + "_scale": torch.zeros(pages, hkv, dtype=torch.uint8, device="cuda") for c in "kv"}
    small = len(x["k_pool"])
    for c in "kv":
        big[c + "_pool"].view(torch.uint8)[pages - small:] = x[c + "_pool"].view(torch.uint8).cuda()
        scale[c + "_scale"][pages - small:] = x[c + "_scale"].cuda()
    y = cuda(x)
    want, _ = run_chunk8(y)
    z = dict(y, **big, **scale, table=torch.where(y["table"] >= 0, y["table"] + (pages - small), -1).int())
    got, st = run_chunk8(z)
    assert st == 0 and same(want, got)
    l1, s1, _ = run_append8(y)
    l2, s2, _ = run_append8(z)
    assert same(l1, l2) and same(s1 + (pages - small) * PAGE, s2)
    assert same(y["v_pool"], z["v_pool"][pages - small:]) and same(y["k_scale"], z["k_scale"][pages - small:])
    del z, big, scale
    pitch, n = 1 << 16, 1 << 15
    wide = torch.zeros(n + 41, pitch, dtype=torch.bfloat16, device="cuda")
    q, k = wide[:, :hq * d].view(n + 41, hq, d), wide[:, 4096:4096 + hkv * d].view(n + 41, hkv, d)
    q[-41:], k[-41:] = x["q"].cuda(), x["k"].cuda()
    cu = torch.tensor([n, n + 40, n + 41], dtype=torch.int32, device="cuda")
    freq, _ = packed.rotary_frequencies(d)
    want = run_rotary(cuda(x), freq)
    packed.mars_rotary(q, k, cu, freq.cuda(), q, k)
    assert same(want[0], q[-41:].contiguous()) and same(want[1], k[-41:].contiguous())


# ----------------------------------------------------------------------------- refusals


def test_bindings_refuse():
    x = cuda(make8([3, 1], 4, 2, 64, [20, 5], seed=90))
    freq = packed.rotary_frequencies(64)[0].cuda()
    q, k, v, cu = x["q"], x["k"], x["v"], x["cu"]
    cache = [x["k_pool"], x["v_pool"], x["k_scale"], x["v_scale"]]
    o, ws = torch.zeros_like(q), torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")

    def chunk(**kw):
        a = dict(q=q, k=k, v=v, cu_seqlens=cu, k_pool=cache[0], v_pool=cache[1], k_scale=cache[2], v_scale=cache[3],
                 block_table=x["table"], seq_lens=x["old"], max_len_hint=30, o=o, workspace=ws)
        packed.mars_attn_chunk_q8(**{**a, **kw})

    def append(**kw):
        a = dict(k=k, v=v, cu_seqlens=cu, seq_lens=x["old"], block_table=x["table"], k_pool=cache[0], v_pool=cache[1],
                 k_scale=cache[2], v_scale=cache[3])
        packed.mars_kv_append_q8(**{**a, **kw})

    def rotary(**kw):
        a = dict(q=q, k=k, cu_seqlens=cu, inv_freq=freq, q_out=torch.zeros_like(q), k_out=torch.zeros_like(k))
        packed.mars_rotary(**{**a, **kw})

    for call in (chunk, append, rotary):
        call()
        for name, t, e in (("cu_seqlens", cu.long(), TypeError), ("cu_seqlens", cu[:0], ValueError),
                           ("k", k.float(), TypeError), ("k", k.cpu(), ValueError), ("k", k[:2], ValueError)):
            with pytest.raises(e):
                call(**{name: t})
    for call in (chunk, append):
        for name, t, e in (("k_pool", cache[0].view(torch.uint8), TypeError), ("v_pool", cache[1][:2], ValueError),
                           ("k_scale", cache[2].float(), TypeError), ("v_scale", cache[3][:, :1], ValueError),
                           ("k_pool", cache[0][..., :32], ValueError), ("block_table", x["table"][0], ValueError),
                           ("v_scale", None, TypeError), ("seq_lens", x["old"][:1], ValueError)):
            with pytest.raises(e):
                call(**{name: t})
    for name, t, e in (("o", o.float(), TypeError), ("workspace", ws[:16], mars.MarsError), ("max_len_hint", 1 << 31, ValueError),
                       ("max_len_hint", -1, mars.MarsError), ("scale", float("inf"), mars.MarsError), ("q", q[:, :3], ValueError)):
        if name == "workspace" and packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, 2, 4, 4, 2, 64, 30) <= 16:
            continue
        with pytest.raises(e):
            chunk(**{name: t})
    lens = x["old"].clone()
    for name, t, e in (("counts", lens.long(), TypeError), ("counts", lens[:1], ValueError), ("slots", lens, ValueError)):
        with pytest.raises(e):
            append(**{name: t})
    both = torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw in (dict(seq_lens=lens, new_lens=lens), dict(counts=lens, new_lens=lens), dict(counts=both[:2], new_lens=both[1:])):
        with pytest.raises(mars.MarsError):
            append(**kw)
    for name, t, e in (("inv_freq", freq.double(), TypeError), ("inv_freq", freq[:7], mars.MarsError), ("inv_freq", freq[:0], mars.MarsError),
                       ("inv_freq", freq[None], ValueError), ("inv_freq", torch.cat([freq, freq]), ValueError),
                       ("factor", float("nan"), mars.MarsError), ("q_out", o.float(), TypeError), ("seq_lens", lens[:1], ValueError)):
        with pytest.raises(e):
            rotary(**{name: t})
    torch.cuda.synchronize()
