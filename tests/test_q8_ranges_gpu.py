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
CODES = 2.0 ** -17                           # q and own k as two e4m3 numbers, relative to a row's largest


def setup(form, seed):
    heads, lens, old = FORMS[form]
    x = make8(lens, *heads, old, seed=seed, tail=1, fused=False)
    return {k: v.clone() if k in "qkv" else v for k, v in x.items()}


def check(x, o, rows, form, own_v=None):
    """Rows of the first sequence, and all of the others, against the definition. The scores are off by what the
    codes of q (2^-17 of its largest element, per element) and of own k lose, each by at most that times the other
    side's magnitudes; a weight then by twice that, relative to it."""
    kv, vv = values(x, "k"), values(x, "v")
    o, cu, g = f64(o), x["cu"].tolist(), x["q"].shape[1] // x["k"].shape[1]
    d = x["q"].shape[2]
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        P = int(x["old"][s])
        e, c = x["table"][s, np.arange(P) // PAGE].numpy().astype(int), np.arange(P) % PAGE
        r = np.array([i for i in rows if i < b - a] if s == 0 else range(min(b - a, 64)), dtype=int)
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
                if form == "middle":
                    of_q = CODES * np.abs(q[r]).max(axis=1, keepdims=True) * np.abs(K).sum(axis=1)
                    of_k = CODES * np.abs(q[r]).sum(axis=1, keepdims=True) * np.abs(K).max(axis=1)
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
    # (of the rows before it only those whose V do not share a power with it)
    check(x, o, [i for i in range(40) if i < j // 16 * 16 or i >= j], form)
