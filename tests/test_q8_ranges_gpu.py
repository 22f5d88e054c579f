"""Attention over the 8-bit cache where the sequences' own rows differ in size: rows that a causal query may
not see, outliers, the ends of the range, infinities and NaN, in every form (needs a GB300)."""
import numpy as np
import pytest
import torch

from packed_util import PAGE, causal_weights, cuda, f64, output_bound
from parity_util import assert_within_bound
from test_q8_gpu import make8, run_chunk8, same, values

pytestmark = pytest.mark.gpu

# (heads, lengths, cached tokens): few rows, a tile of 128 (token, head) rows, many
FORMS = {"few": ((14, 2, 64), [16], [90]), "middle": ((24, 1, 128), [40, 16, 5], [200, 37, 0]),
         "many": ((28, 4, 128), [1400, 16], [300, 5])}
forms = pytest.mark.parametrize("form", FORMS)

MOST_VALUE = (1 + 127 / 128) * 2.0 ** 87     # the largest bf16 below 2^88: larger own values count as this
# q and own k as two e4m3 numbers, relative to a row's largest: 2^-17 over a power of its own, and 16 own keys share
# one while their largest are within a factor of 2^3
CODES_Q, CODES_K = 2.0 ** -17, 2.0 ** -14


def setup(form, seed):
    heads, lens, old = FORMS[form]
    x = make8(lens, *heads, old, seed=seed, tail=1, fused=False)
    return {k: v.clone() if k in "qkv" else v for k, v in x.items()}


def check(x, o, rows, form, own_v=None):
    """Rows of the first sequence, and all of the others, against the definition. The scores are off by what the
    codes of q and of own k lose (above, per element), each by at most that times the other
    side's magnitudes; a weight then by twice that, relative to it."""
    kv, vv = values(x, "k"), values(x, "v")
    o, cu, g = f64(o), x["cu"].tolist(), x["q"].shape[1] // x["k"].shape[1]
    d = x["q"].shape[2]
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        P = int(x["old"][s])
        e, c = x["table"][s, np.arange(P) // PAGE].numpy().astype(int), np.arange(P) % PAGE
        r = np.array([i for i in rows if i < b - a] if s == 0 else range(min(b - a, 64)), dtype=int)
        if b == a:
            continue
        for u in range(x["k"].shape[1]):
            K = np.concatenate([kv[e, u, c].reshape(-1, d), f64(x["k"][a:b, u])])
            own = f64(x["v"][a:b, u])
            if form != "many":
                own = np.where(np.isfinite(own), np.clip(own, -MOST_VALUE, MOST_VALUE), own)
            V = np.concatenate([vv[e, u, c].reshape(-1, d), own])
            for h in range(u * g, u * g + g):
                q = f64(x["q"][a:b, h])
                w = causal_weights(q, K)[r]
                ref = w @ V
                seen = np.arange(len(K)) <= r[:, None] + P
                off = np.zeros(len(r))
                if form == "middle" or (form == "many" and s > 0):     # (16 rows: a tile of 128 (token, head) rows)
                    of_q = CODES_Q * np.abs(q[r]).max(axis=1, keepdims=True) * np.abs(K).sum(axis=1)
                    of_k = CODES_K * np.abs(q[r]).sum(axis=1, keepdims=True) * np.abs(K).max(axis=1)
                    off = 2 / np.sqrt(d) * np.where(seen, of_q + of_k, 0).max(axis=1)
                bound = output_bound(w, V, ref) + off[:, None] * (w @ np.abs(V))
                assert_within_bound(o[a:b, h][r], ref, bound, f"sequence {s} head {h}")


@pytest.mark.parametrize("power", [48, 79, 87, 97, 120])
@forms
def test_large_own_values(form, power):
    """One own V row of up to the largest size: no row that may not see it notices, one that does gets its share,
    and the weights of the other keys are not lost beside it, whatever their pages' scales."""
    x = setup(form, 100 + power)
    j = 9 if form == "few" else 25
    x["v"][j] *= 2.0 ** power
    for lp in range(5):
        x["v_scale"][x["table"][0, lp]] = 87 + 8 * lp
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check(x, o, range(40), form)


@pytest.mark.parametrize("power", [6, 10, 14, 20, 60])
@pytest.mark.parametrize("what", ["k", "v"])
@forms
def test_later_own_rows_take_nothing_from_earlier_ones(form, what, power):
    """The last of 16 own rows is far larger than the others: the rows before it do not see it."""
    x = setup(form, 200 + power)
    x[what][15] *= 2.0 ** power
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check(x, o, range(15), form)
    if what == "v":
        check(x, o, range(15, 40), form)
    elif power <= 20:
        # (scores of 2^60 are rounded by up to 2^36, and exp2 of that is beyond 32 bits)
        assert torch.isfinite(o).all()


@pytest.mark.parametrize("power", [4, 8, 12])
@forms
def test_one_large_element_of_a_query_or_key(form, power):
    """An element of every q row or own k row, of a dimension where the other side is small, so that the scores stay
    of the size that the bound of their fp32 sums knows."""
    for what, other in (("q", "k"), ("k", "q")):
        x = setup(form, 300 + power)
        x[what][:, :, 5] *= 2.0 ** power
        x[other][:, :, 5] *= 2.0 ** -power
        if other == "k":
            raw = x["k_pool"].float()
            raw[..., 5] *= 2.0 ** -power
            x["k_pool"] = raw.to(torch.float8_e4m3fn)
        o, st = run_chunk8(cuda(x))
        assert st == 0
        check(x, o, range(40), form)


@pytest.mark.parametrize("power", [-30, 30])
@forms
def test_sizes_near_the_ends_of_the_powers(form, power):
    """q and k of sizes whose product is ordinary, own rows and cached ones alike; V of any size."""
    x = setup(form, 400 + power)
    x["q"] *= 2.0 ** power
    x["k"] *= 2.0 ** -power
    x["v"] *= 2.0 ** -power
    for c in "kv":
        x[c + "_scale"] = (x[c + "_scale"].int() - power).to(torch.uint8)
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check(x, o, range(40), form)


@forms
def test_own_rows_of_zeros(form):
    x = setup(form, 500)
    x["v"][3:8] = 0
    x["k"][5:9] = 0
    x["q"][2] = 0
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check(x, o, range(40), form)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")], ids=str)
@forms
def test_infinities_and_nan_of_own_rows_are_not_lost(form, bad):
    """They reach the rows that see them, and no other sequence."""
    heads = FORMS[form][0]
    j = 9 if form == "few" else 20
    clean = run_chunk8(cuda(setup(form, 600)))[0]
    n = FORMS[form][1][0]
    x = setup(form, 600)
    x["v"][j, 0, 7] = bad
    o, st = run_chunk8(cuda(x))
    assert st == 0
    group = slice(0, heads[0] // heads[1])
    assert not torch.isfinite(o[j:n, group, 7].float()).any()
    o[:n, group, 7] = clean[:n, group, 7]
    assert same(o, clean)
    x = setup(form, 600)
    x["k"][j, 0, 7] = bad
    o, st = run_chunk8(cuda(x))
    assert st == 0
    # NaN or +infinity as a score (where it is -infinity the key has no weight)
    hit = x["q"][j:n, group, 7].float() * bad
    hit = ~(hit < 0)
    assert torch.isnan(o[j:n, group][hit.cuda()]).all()
    if heads[1] > 1:
        assert same(o[:, heads[0] // heads[1]:], clean[:, heads[0] // heads[1]:])
    assert same(o[n:], clean[n:])


@pytest.mark.parametrize("form", ["few", "middle"])
def test_weights_keep_what_f16_has(form):
    """Relative to the norm. The result's rounding to bf16 gives what rounding the exact one gives (r, over so many
    elements that chance moves it by less than 3 %). Rounding the weights to f16 adds independent errors of at most
    2^-11 of each p v, whose squares sum to a third of 2^-22 (sum p^2 v^2); twice that leaves room for scores and
    sums in 32 bits and the codes of q, each far below it. Weights in bf16 would add eight times as much."""
    heads, batch = FORMS[form][0], 24
    lens, old = ([2] * batch if form == "few" else [16] * batch), [500 + 31 * i for i in range(batch)]
    x = make8(lens, *heads, old, seed=700)
    o, st = run_chunk8(cuda(x))
    assert st == 0
    kv, vv = values(x, "k"), values(x, "v")
    o, cu, g, d = f64(o), x["cu"].tolist(), heads[0] // heads[1], heads[2]
    err = rounding = spread = 0.0
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        P = old[s]
        e, c = x["table"][s, np.arange(P) // PAGE].numpy().astype(int), np.arange(P) % PAGE
        for u in range(heads[1]):
            K = np.concatenate([kv[e, u, c].reshape(-1, d), f64(x["k"][a:b, u])])
            V = np.concatenate([vv[e, u, c].reshape(-1, d), f64(x["v"][a:b, u])])
            for h in range(u * g, u * g + g):
                w = causal_weights(f64(x["q"][a:b, h]), K)
                ref = w @ V
                err += ((o[a:b, h] - ref) ** 2).sum()
                rounding += ((f64(torch.from_numpy(ref).to(torch.bfloat16)) - ref) ** 2).sum()
                spread += (w ** 2 @ V ** 2).sum()
    assert err <= 1.03 ** 2 * rounding + 2 * 2.0 ** -22 / 3 * spread, (err / rounding, spread / rounding)


MIXED = [((24, 1, 128), [(7 * i) % 21 for i in range(60)], [0] * 60),
         ((24, 1, 128), [16] * 70, [(37 * i) % 150 for i in range(70)]),
         ((28, 4, 128), [170, 130, 17], [40, 0, 300]), ((130, 1, 64), [300, 520, 1], [0, 140, 9]),
         ((96, 1, 64), [140, 3, 260], [1000, 0, 5])]


@pytest.mark.parametrize("heads, lens, old", MIXED, ids=lambda v: str(v)[:24])
def test_rows_of_all_sizes_in_many_items(heads, lens, old):
    """Own rows of sizes far apart wherever they stand: items of nothing else, of several own tiles, one after another
    in a CTA, and beside rows of one size."""
    x = make8(lens, *heads, old, seed=800, tail=1, fused=False)
    x = {k: v.clone() if k in "qkv" else v for k, v in x.items()}
    rng = np.random.default_rng(801)
    n, hkv = x["k"].shape[:2]
    for c, most in (("k", 14), ("v", 20)):
        down = rng.integers(0, most + 1, size=(n, hkv, 1)) * (rng.random((n, 1, 1)) < 0.6)
        down[: n // 3] = 0
        x[c] *= torch.from_numpy(np.exp2(-down.astype(float))).to(torch.bfloat16)
    o, st = run_chunk8(cuda(x))
    assert st == 0
    check(x, o, range(max(lens)), "middle")
    for _ in range(3):
        again, _ = run_chunk8(cuda(x))
        assert same(o, again)
