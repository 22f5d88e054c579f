"""Packed sequences on the CPU: what pins the oracle, and what the entry points refuse."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from block_masked_token_gb300 import mars, packed
from packed_util import PAGE, f64, make


# ---------------------------------------------------------------------------- the oracle

def test_packed_is_the_clean_stream_of_the_dual_form():
    """One sequence is the clean half of the dual-stream attention, statistics included."""
    x = make([11], 4, 2, 64, seed=1)
    q, k, v = (f64(x[c]) for c in "qkv")
    two = lambda t: np.concatenate([t, np.zeros_like(t)])[None]      # noqa: E731
    o, lse = oracle.attn_packed(q, k, v, [0, 11])
    np.testing.assert_allclose(o, oracle.attn_dual_stream(two(q), two(k), two(v), 11, 4)[0, :11], atol=1e-13)
    np.testing.assert_allclose(lse, oracle.attn_dual_stream_lse(two(q), two(k), 11, 4)[0, :, :11], atol=1e-12)


def test_packed_sequences_do_not_see_each_other():
    x = make([5, 0, 7], 4, 2, 64, seed=2)
    q, k, v = (f64(x[c]) for c in "qkv")
    o, lse = oracle.attn_packed(q, k, v, x["cu"].numpy())
    a, la = oracle.attn_packed(q[:5], k[:5], v[:5], [0, 5])
    b, lb = oracle.attn_packed(q[5:], k[5:], v[5:], [0, 7])
    assert (o == np.concatenate([a, b])).all() and (lse == np.concatenate([la, lb], 1)).all()
    assert (o[0] == v[0].repeat(2, 0)).all()           # one key: its value


def test_chunk_is_the_tail_of_the_whole_prompt():
    x = make([40, 9], 4, 2, 64, seed=3, old=[0, 0])
    q, k, v = (f64(x[c]) for c in "qkv")
    whole, _ = oracle.attn_packed(q, k, v, x["cu"].numpy())
    first = np.array([0, 33, 35])                      # 33 and 2 rows cached, 7 and 7 new
    rows = np.r_[0:33, 40:42]
    kp, vp, lens, _ = oracle.kv_append(k[rows], v[rows], first, [0, 0], x["table"].numpy(),
                                       f64(x["k_pool"]), f64(x["v_pool"]), PAGE)
    assert lens.tolist() == [33, 2]
    rest = np.r_[33:40, 42:49]
    o = oracle.attn_chunk(q[rest], k[rest], v[rest], [0, 7, 14], kp, vp, x["table"].numpy(), lens, PAGE)
    np.testing.assert_allclose(o, whole[rest], atol=1e-13)


def test_append_is_the_commit_of_every_row():
    x = make([6, 6], 4, 2, 64, seed=4, old=[13, 40])
    k, v = f64(x["k"]), f64(x["v"])
    got = oracle.kv_append(k, v, [0, 6, 12], [13, 40], x["table"].numpy(), f64(x["k_pool"]), f64(x["v_pool"]), PAGE)
    want = oracle.kv_commit(k.reshape(2, 6, 2, 64), v.reshape(2, 6, 2, 64), [6, 6], [13, 40],
                            x["table"].numpy(), f64(x["k_pool"]), f64(x["v_pool"]), PAGE)
    for a, b in zip(got, want):
        assert (a == b.reshape(a.shape)).all()


def test_packed_gradient_matches_differences():
    rng = np.random.default_rng(5)
    q, k, v, do = (rng.normal(size=(9, h, 8)) for h in (4, 2, 2, 4))
    cu = [0, 3, 3, 9]
    loss = lambda q, k, v: float((oracle.attn_packed(q, k, v, cu)[0] * do).sum())      # noqa: E731
    grads = oracle.attn_packed_grad(q, k, v, do, cu)
    for which in range(3):
        for _ in range(25):
            at = tuple(rng.integers(0, m) for m in (q, k, v)[which].shape)
            args = [q.copy(), k.copy(), v.copy()]
            args[which][at] += 1e-5
            up = loss(*args)
            args[which][at] -= 2e-5
            assert abs((up - loss(*args)) / 2e-5 - grads[which][at]) < 1e-8


def test_packed_gradient_matches_autograd():
    x = make([12, 1, 30], 4, 2, 64, seed=6)
    q, k, v = (x[c].double().detach().requires_grad_() for c in "qkv")
    out = []
    for a, b in ((0, 12), (12, 13), (13, 43)):
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b].repeat_interleave(2, 1)) / 8.0
        s = s.masked_fill(torch.ones(b - a, b - a).triu(1).bool(), -torch.inf).softmax(-1)
        out.append(torch.einsum("hij,jhd->ihd", s, v[a:b].repeat_interleave(2, 1)))
    (torch.cat(out) * x["do"].double()).sum().backward()
    got = oracle.attn_packed_grad(f64(x["q"]), f64(x["k"]), f64(x["v"]), f64(x["do"]), x["cu"].numpy())
    for a, b in zip(got, (q, k, v)):
        np.testing.assert_allclose(a, b.grad.numpy(), atol=1e-12)


# ------------------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(mars._LIB_PATH):
        from block_masked_token_gb300.build import build_library
        build_library()
    return mars.lib()


P, BAD = ctypes.c_void_p(4096), ctypes.c_void_p(4100)


def attn_packed(L, q=P, k=P, v=P, cu=P, o=P, lse=None, batch=2, total=40, hq=4, hkv=2, d=64,
                strides=(512, 512, 512), scale=0.0, ws=P, ws_bytes=1 << 30):
    return L.mars_attn_packed(q, k, v, cu, o, lse, batch, total, hq, hkv, d, *strides, scale, ws,
                              ws_bytes, None, None)


def attn_chunk(L, q=P, k=P, v=P, cu=P, kp=P, vp=P, pages=10, table=P, max_pages=4, lens=P, hint=64,
               o=P, batch=2, total=40, hq=4, hkv=2, d=64, page=16, strides=(512, 512, 512),
               scale=0.0, ws=P, ws_bytes=1 << 30):
    return L.mars_attn_chunk(q, k, v, cu, kp, vp, pages, table, max_pages, lens, hint, o, batch,
                             total, hq, hkv, d, page, *strides, scale, ws, ws_bytes, None, None)


def append(L, k=P, v=P, cu=P, lens=P, new=None, table=P, max_pages=4, kp=P, vp=P, pages=10,
           slots=None, batch=2, total=40, hkv=2, d=64, page=16, strides=(512, 512)):
    return L.mars_kv_append(k, v, cu, lens, new, table, max_pages, kp, vp, pages, slots, batch,
                            total, hkv, d, page, *strides, None, None)


def grad(L, q=P, k=P, v=P, o=P, d_o=P, lse=P, cu=P, dq=P, dk=P, dv=P, batch=2, total=40, hq=4,
         hkv=2, d=64, strides=(512,) * 6, scale=0.0, ws=P, ws_bytes=1 << 30):
    return L.mars_attn_packed_grad(q, k, v, o, d_o, lse, cu, dq, dk, dv, batch, total, hq, hkv, d,
                                   *strides, scale, ws, ws_bytes, None, None)


@pytest.mark.parametrize("change, code", [
    *[({n: None}, mars.EINVAL) for n in ("q", "v", "o", "d_o", "lse", "cu", "dq", "dk", "dv", "ws")],
    *[({n: BAD}, mars.EALIGN) for n in ("k", "o", "d_o", "dq", "dv", "ws")],
    ({"strides": (512, 512, 512, 248, 512, 512)}, mars.EINVAL),
    ({"strides": (512, 512, 512, 512, 512, 132)}, mars.EALIGN), ({"hq": 3}, mars.EINVAL),
    ({"d": 32}, mars.EUNSUPPORTED), ({"total": -2}, mars.EINVAL), ({"ws_bytes": 64}, mars.ENOSPACE),
    ({"scale": float("inf")}, mars.EINVAL), ({"total": 0}, mars.OK), ({"batch": 0}, mars.OK),
    # more tiles times heads, or blocks of rows, than 32 bits count
    ({"batch": 1 << 29, "ws_bytes": 1 << 62}, mars.EUNSUPPORTED),
    ({"batch": 1 << 28, "hq": 2, "ws_bytes": 1 << 62}, mars.EUNSUPPORTED)], ids=str)
def test_gradient_refusals(L, change, code):
    assert grad(L, **change) == code


SHARED = [({"q": None}, mars.EINVAL), ({"cu": None}, mars.EINVAL), ({"o": None}, mars.EINVAL),
          ({"k": BAD}, mars.EALIGN), ({"o": BAD}, mars.EALIGN), ({"ws": BAD}, mars.EALIGN),
          ({"batch": -1}, mars.EINVAL), ({"total": -1}, mars.EINVAL),
          ({"total": 0x7fffffff}, mars.EINVAL), ({"hq": 3}, mars.EINVAL), ({"hkv": 0}, mars.EINVAL),
          ({"d": 96}, mars.EUNSUPPORTED), ({"strides": (248, 512, 512)}, mars.EINVAL),
          ({"strides": (512, 127, 512)}, mars.EINVAL), ({"strides": (512, 512, 132)}, mars.EALIGN),
          ({"scale": float("inf")}, mars.EINVAL), ({"batch": 0}, mars.OK), ({"total": 0}, mars.OK)]


@pytest.mark.parametrize("change, code", SHARED, ids=str)
def test_attention_refusals(L, change, code):
    assert attn_packed(L, **change) == code
    assert attn_chunk(L, **change) == code


@pytest.mark.parametrize("change, code", [
    ({"lens": None}, mars.EINVAL), ({"table": None}, mars.EINVAL), ({"kp": None}, mars.EINVAL),
    ({"vp": BAD}, mars.EALIGN), ({"hint": -1}, mars.EINVAL), ({"max_pages": -1}, mars.EINVAL),
    ({"pages": -1}, mars.EINVAL), ({"pages": 1 << 27}, mars.EINVAL), ({"page": 32}, mars.EUNSUPPORTED),
    ({"total": 1, "batch": 1, "hint": 100000, "ws_bytes": 16}, mars.ENOSPACE),
    ({"total": 1, "batch": 1, "hint": 100000, "ws": None}, mars.EINVAL)], ids=str)
def test_chunk_refusals(L, change, code):
    assert attn_chunk(L, **change) == code


@pytest.mark.parametrize("change, code", [
    ({"k": None}, mars.EINVAL), ({"vp": None}, mars.EINVAL), ({"lens": None}, mars.EINVAL),
    ({"cu": None}, mars.EINVAL), ({"table": None}, mars.EINVAL), ({"new": P}, mars.EINVAL),
    ({"v": BAD}, mars.EALIGN), ({"kp": BAD}, mars.EALIGN), ({"strides": (512, 100)}, mars.EINVAL),
    ({"strides": (132, 512)}, mars.EALIGN), ({"d": 32}, mars.EUNSUPPORTED), ({"page": 8}, mars.EUNSUPPORTED),
    ({"pages": -1}, mars.EINVAL), ({"max_pages": -1}, mars.EINVAL), ({"batch": -1}, mars.EINVAL),
    ({"batch": 0}, mars.OK)], ids=str)
def test_append_refusals(L, change, code):
    assert append(L, **change) == code


def test_workspace_sizes(L):
    size = packed.mars_packed_workspace_bytes
    assert size(99, 1, 10) == 0 and size(packed.OP_ATTN_CHUNK, 1, 10, 3, 2, 64, 9000) == 0
    assert size(packed.OP_ATTN_CHUNK, 1, 1, 28, 4, 128, -1) == 0
    assert size(packed.OP_ATTN_CHUNK, 1, 1, 28, 4, 128, 8192) > 0      # one token: split
    assert size(packed.OP_ATTN_CHUNK, 0, 0, 28, 4, 128, 8192) == 0


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_bindings_refuse_host_tensors(L):
    q, k, ws = bf(4, 2, 64), bf(4, 1, 64), torch.zeros(64, dtype=torch.uint8)
    pool = bf(4, 1, 16, 64)
    for call in (lambda: packed.mars_attn_packed(q, k, k, i32(2), q, ws),
                 lambda: packed.mars_attn_packed_grad(q, k, k, q, q, torch.zeros(2, 4), i32(2), q, k, k, ws),
                 lambda: packed.mars_attn_chunk(q, k, k, i32(2), pool, pool, i32(1, 4), i32(1), 9, q, ws),
                 lambda: packed.mars_kv_append(k, k, i32(2), i32(1), i32(1, 4), pool, pool)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("t, match", [
    (bf(4, 64, 2).transpose(1, 2), "contiguous"), (bf(4, 2, 128)[:, :, ::2], "contiguous"),
    (bf(4, 2 * 64 + 4)[:, :128].view(4, 2, 64), "pitch"), (bf(1, 2, 64).expand(4, 2, 64), "pitch"),
    (bf(5, 2, 64), "shape")], ids=["heads", "elements", "pitch", "broadcast", "shape"])
def test_row_layouts_that_are_refused(monkeypatch, t, match):
    class Host:                       # a host tensor that says it is on the GPU
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, n):
            return getattr(self.t, n)

        def get_device(self):
            return 0

    monkeypatch.setattr(packed, "torch", type("T", (), {"Tensor": Host}))
    with pytest.raises(ValueError, match=match):
        packed._rows(Host(t), "q", (4, 2, 64), 0)
    with pytest.raises(ValueError, match="cuda:0"):
        packed._rows(Host(bf(4, 2, 64)), "q", (4, 2, 64), 1)
    assert packed._rows(Host(bf(4, 6, 64)[:, 1:3]), "q", (4, 2, 64), 0)[1] == 384
    assert packed._rows(Host(bf(1, 2, 64)), "q", (1, 2, 64), 0)[1] == 128


@pytest.mark.parametrize("batch, total, hq, hkv, d", [(1, 1, 4, 2, 64), (32, 32, 28, 4, 128), (3, 4000, 28, 4, 128)])
def test_workspace_of_the_largest_hints(L, batch, total, hq, hkv, d):
    """The splits of the longest lists that a hint can name: their number, and with it the
    workspace, no longer changes there."""
    sizes = {packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK, batch, total, hq, hkv, d, h)
             for h in (1 << 30, (1 << 31) - 129, (1 << 31) - 128, (1 << 31) - 127, (1 << 31) - 1)}
    assert len(sizes) == 1 and sizes.pop() > 0


def test_rows_wider_than_the_kernels_count_are_refused(L):
    """The append counts the 16-byte vectors of 16 rows in 31 bits: rows of up to 2^29 elements."""
    wide = (1 << 23) + 1
    assert append(L, hkv=wide, pages=1, batch=0, strides=(64 * wide,) * 2) == mars.EINVAL
    assert append(L, hkv=wide - 1, pages=1, batch=0, strides=(64 * wide,) * 2) == mars.OK
    for call in (attn_packed, attn_chunk, grad):
        assert call(L, hq=wide, hkv=1, batch=0) == mars.EINVAL
        assert call(L, hq=wide - 1, hkv=1, batch=0) == mars.OK


@pytest.mark.parametrize("at", [4092, 4096, 4100])
def test_append_refuses_new_lengths_over_the_old_ones(L, at):
    assert append(L, new=ctypes.c_void_p(at)) == mars.EINVAL


def test_bindings_refuse_counts_beyond_31_bits(L):
    """ctypes would pass on their low 32 bits."""
    size, big = packed.mars_packed_workspace_bytes, 1 << 32
    good = dict(batch=1, total=1, hq=28, hkv=4, d=128, max_len=8192)
    assert size(packed.OP_ATTN_CHUNK, **good) > 0
    for name in good:
        assert size(packed.OP_ATTN_CHUNK, **{**good, name: good[name] + big}) == 0
        assert size(packed.OP_ATTN_CHUNK, **{**good, name: good[name] - big}) == 0
    meta = dict(device="meta")
    with pytest.raises(ValueError, match="31 bits"):
        packed._table(torch.empty(1, big + 5, dtype=torch.int32, **meta), 1, 0)
    with pytest.raises(ValueError, match="31 bits"):
        packed._rows(torch.empty(big + 5, 1, 64, dtype=torch.bfloat16, **meta), "k", (big + 5, 1, 64), 0)
    with pytest.raises(ValueError, match="31 bits"):
        packed._batch(torch.empty(big + 5, dtype=torch.int32, **meta), 0)
