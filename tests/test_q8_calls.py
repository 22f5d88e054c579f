"""Rotary positions and the 8-bit cache on the host: the C form of their calls (csrc/packed_calls.c)
with entry points that record their arguments, what it declines, and the refusals of the library,
which come before anything is launched."""
import ctypes
import math

import pytest
import torch

from block_masked_token_gb300 import mars, packed
from test_packed_calls import STREAM, Host, bf, calls, i32  # noqa: F401  (calls: the fixture)

NAMES = ("mars_rotary", "mars_kv_append_q8", "mars_attn_chunk_q8")


@pytest.fixture()
def calls8(calls):                                    # noqa: F811
    module, _ = calls
    made, keep = [], []

    def recorder(name):
        def record(*a):
            made.append(a)
            return 7
        keep.append(ctypes.CFUNCTYPE(ctypes.c_int, *getattr(mars.lib(), name).argtypes)(record))
        return ctypes.cast(keep[-1], ctypes.c_void_p).value

    module.setup_q8(torch.float8_e4m3fn, *map(recorder, NAMES))
    yield module, made
    keep.clear()                          # (which has held the entry points until here)


def e4m3(*shape):
    return Host(torch.zeros(*shape, dtype=torch.uint8).view(torch.float8_e4m3fn))


def u8(*shape):
    return Host(torch.zeros(*shape, dtype=torch.uint8))


def arguments(name):
    """Positional arguments of the C form, what the library has to get, and which may be None."""
    total, hq, hkv, d, batch, pages, width = 7, 4, 2, 64, 3, 9, 5
    qkv = torch.zeros(total, hq + 2 * hkv, d, dtype=torch.bfloat16)
    q, k, v = (Host(t) for t in qkv.split([hq, hkv, hkv], dim=1))
    cu, lens, counts, new, slots = i32(batch + 1), i32(batch), i32(batch), i32(batch), i32(total)
    table, status, o = i32(batch, width), i32(1), bf(total, hq, d)
    cache = [e4m3(pages, hkv, 16, d), e4m3(pages, hkv, 16, d), u8(pages, hkv), u8(pages, hkv)]
    p = lambda *ts: tuple(t.data_ptr() for t in ts)                  # noqa: E731
    wide = (hq + 2 * hkv) * d
    if name == "rotary":
        freq, ko = Host(torch.zeros(24)), bf(total, hkv, d)
        return ([q, k, cu, freq, o, ko, lens, True, 1.5, False, status],
                (*p(q, k, cu, lens, freq, o, ko), batch, total, hq, hkv, d, 48, 1, 0, 1.5, wide, wide, hq * d,
                 hkv * d, *p(status), STREAM), (6, 10))
    if name == "kv_append_q8":
        return ([k, v, cu, *cache, table, lens, counts, new, slots, status, 16],
                (*p(k, v, cu, lens, counts, new, table), width, *p(*cache), pages, *p(slots), batch, total, hkv, d,
                 16, wide, wide, *p(status), STREAM), (9, 10, 11, 12))
    ws = u8(300)
    return ([q, k, v, cu, *cache, table, lens, 99, o, ws, status, 0.25, 16],
            (*p(q, k, v, cu, *cache), pages, *p(table), width, *p(lens), 99, *p(o), batch, total, hq, hkv, d, 16,
             wide, wide, wide, 0.25, *p(ws), 300, *p(status), STREAM), (13,))


@pytest.mark.parametrize("name", [n[5:] for n in NAMES])
def test_arguments_reach_the_library(calls8, name):
    module, made = calls8
    given, want, optional = arguments(name)
    assert getattr(module, name)(*given) == 7
    assert made == [want]
    for i in optional:
        assert getattr(module, name)(*given[:i], None, *given[i + 1:]) == 7
        assert sum(a is None for a in made[-1]) == 1


@pytest.mark.parametrize("name", [n[5:] for n in NAMES])
def test_every_wrong_argument_is_declined(calls8, name):
    """Each argument in turn: of another type, shape, device or layout, or missing."""
    module, made = calls8
    call = getattr(module, name)
    given, _, optional = arguments(name)
    for i, x in enumerate(given):
        bad = [object(), "x"]
        if isinstance(x, Host):
            t = x.t
            other = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.to(torch.float64)
            bad += [Host(other), Host(t, device=1), Host(t, device=-1), Host(t[None])]
            if not (name == "attn_chunk_q8" and i == 12):            # any amount of scratch
                bad.append(Host(torch.zeros([s + 1 for s in t.shape]).to(t.dtype)))
            if not (t.dim() == 1 and t.shape[0] == 1):               # one element has no stride to be wrong
                bad.append(Host(torch.zeros([2 * s for s in t.shape]).to(t.dtype)[
                    tuple(slice(0, None, 2) for _ in t.shape)]))
            if name == "rotary" and i == 3:
                bad[-2] = Host(torch.zeros(33))                      # more than d / 2 frequencies
        elif isinstance(x, bool):
            bad += [1, 0.0, None]
        elif isinstance(x, float):
            bad += [None, 1]
        elif x == 16:
            bad += [0, -1, 1 << 31, 32, 1 << 70]
        elif x == 99:
            bad += [-1, 1 << 31, 1 << 70, 9.0]
        for y in bad:
            assert call(*given[:i], y, *given[i + 1:]) is None, (i, y)
        if i not in optional:
            assert call(*given[:i], None, *given[i + 1:]) is None, i
    assert not made
    assert call(*given[:-1]) is None and call() is None and not made


@pytest.mark.parametrize("n", [0, 3, 5])
def test_setup_takes_four(calls8, n):
    with pytest.raises(TypeError):
        calls8[0].setup_q8(*[0] * n)


def P(v=16):
    return ctypes.c_void_p(v)


def code(name, base, **kw):
    """The library's return code for `base` with some arguments replaced, by position."""
    a = list(base)
    for i, x in kw.items():
        a[int(i[1:])] = x
    return getattr(mars.lib(), name)(*a)


def test_rotary_refusals():
    # q k cu lens freq q_out k_out | batch total hq hkv d rot interleaved inverse | factor | pitches
    a = [P()] * 7 + [2, 9, 4, 2, 64, 64, 0, 0, 1.0, 256, 128, 256, 128, None, None]
    c = lambda **kw: code("mars_rotary", a, **kw)                    # noqa: E731
    assert c(_7=0) == mars.OK and c(_8=0) == mars.OK
    for i in (0, 1, 2, 4, 5, 6):
        assert c(**{f"_{i}": None}) == mars.EINVAL
    for i in (0, 1, 5, 6):
        assert c(**{f"_{i}": P(24)}) == mars.EALIGN
    for rot, want in ((0, mars.EINVAL), (-16, mars.EINVAL), (80, mars.EINVAL), (8, mars.EUNSUPPORTED),
                      (24, mars.EUNSUPPORTED)):
        assert c(_12=rot) == want
    for f in (math.nan, math.inf, -math.inf):
        assert c(_15=f) == mars.EINVAL
    assert c(_11=96) == mars.EUNSUPPORTED and c(_9=3) == mars.EINVAL and c(_7=-1) == mars.EINVAL
    for i, pitch in ((16, 255), (16, 248), (17, 132), (18, 0), (19, 120), (19, -128)):
        assert c(**{f"_{i}": pitch}) < 0
    # in place with another pitch
    assert c(_5=P(32), _6=P(48), _0=P(32), _18=264) == mars.EINVAL
    assert c(_5=P(32), _6=P(48), _1=P(48), _19=136) == mars.EINVAL


def test_append_refusals():
    # k v cu lens counts new_lens table | width | pools scales | pages slots batch total hkv d page pitches
    a = [P(), P(), P(), P(1024), P(2048), P(4096), P(), 4, P(), P(), P(), P(), 9, None, 2, 9, 2, 64, 16, 128, 128, None,
         None]
    c = lambda **kw: code("mars_kv_append_q8", a, **kw)              # noqa: E731
    assert c(_14=0) == mars.OK
    for i in (0, 1, 2, 3, 6, 8, 9, 10, 11):
        assert c(**{f"_{i}": None}) == mars.EINVAL
    for i in (0, 1, 8, 9):
        assert c(**{f"_{i}": P(24)}) == mars.EALIGN
    assert c(_18=8) == mars.EUNSUPPORTED and c(_17=80) == mars.EUNSUPPORTED
    for i in (7, 12, 14, 15):
        assert c(**{f"_{i}": -1}) == mars.EINVAL
    assert c(_16=0) == mars.EINVAL and c(_12=1 << 30) == mars.EINVAL  # more rows than 32 bits count
    assert c(_5=P(1024)) == mars.EINVAL and c(_5=P(1028)) == mars.EINVAL and c(_5=P(2044)) == mars.EINVAL
    for i, pitch in ((19, 120), (19, 132), (20, 0)):
        assert c(**{f"_{i}": pitch}) < 0


def test_chunk_refusals():
    # q k v cu pools scales | pages table width lens hint o | batch total hq hkv d page pitches | scale ws bytes
    a = [P()] * 8 + [9, P(), 4, P(), 100, P(), 2, 9, 4, 2, 64, 16, 256, 128, 128, 0.0, P(256), 1 << 40, None, None]
    c = lambda **kw: code("mars_attn_chunk_q8", a, **kw)             # noqa: E731
    assert c(_14=0) == mars.OK and c(_15=0) == mars.OK
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 11, 13):
        assert c(**{f"_{i}": None}) == mars.EINVAL
    for i in (0, 1, 2, 4, 5, 13):
        assert c(**{f"_{i}": P(24)}) == mars.EALIGN
    assert c(_19=32) == mars.EUNSUPPORTED and c(_18=80) == mars.EUNSUPPORTED
    for i in (8, 10, 12, 14, 15):
        assert c(**{f"_{i}": -1}) == mars.EINVAL
    assert c(_16=3) == mars.EINVAL and c(_23=math.inf) == mars.EINVAL and c(_8=1 << 30) == mars.EINVAL
    for i, pitch in ((20, 248), (20, 260), (21, 0), (22, 120)):
        assert c(**{f"_{i}": pitch}) < 0
    need = packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, 2, 9, 4, 2, 64, 5000)
    assert need > 0
    assert c(_12=5000, _25=need - 1) == mars.ENOSPACE and c(_12=5000, _24=None) == mars.EINVAL


@pytest.mark.parametrize("hq, hkv, d", [(28, 4, 128), (4, 2, 64), (96, 1, 64), (16, 16, 128)])
def test_workspace_sizes(hq, hkv, d):
    """Sizes of any arguments fit, and grow with none of the keys beyond what parts there can be."""
    size = lambda *a: packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, *a)   # noqa: E731
    for batch, total in ((1, 1), (3, 3), (3, 20), (64, 64), (500, 500), (7, 4000), (1, 1 << 20)):
        sizes = [size(batch, total, hq, hkv, d, n) for n in (0, 100, 1000, 20000, 1 << 30, 2 ** 31 - 1)]
        assert all(0 <= s < 1 << 40 for s in sizes) and sizes[-1] > 0
    assert size(0, 1, hq, hkv, d, 1) == size(1, 0, hq, hkv, d, 1) == size(2, 9, hq, hkv, 96, 100) == 0


def test_more_sequences_than_a_grid_has_places():
    """2^31 - 1 sequences of as many rows: refused before anything is launched, and sizes that do not wrap."""
    big = 2 ** 31 - 1
    rotary = [P()] * 7 + [big, big, 1, 1, 64, 64, 0, 0, 1.0, 64, 64, 64, 64, None, None]
    append = [P(), P(), P(), P(), None, None, P(), 4, P(), P(), P(), P(), 9, None, big, big, 1, 64, 16, 64, 64, None, None]
    chunk = [P()] * 8 + [9, P(), 4, P(), 100, P(), big, big, 1, 1, 64, 16, 64, 64, 64, 0.0, P(256), (1 << 63) - 1, None,
                         None]
    for name, a in (("mars_rotary", rotary), ("mars_kv_append_q8", append), ("mars_attn_chunk_q8", chunk)):
        assert code(name, a) in (mars.EINVAL, mars.EUNSUPPORTED)
    for batch, total in ((big, big), (big - 1, 1), (1, big - 1), (1 << 20, 1 << 30)):
        size = packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, batch, total, 1, 1, 64, 100)
        assert 0 <= size < 1 << 50


def fits(batch, total, hq, hkv, d, hint, ws_bytes):
    """Whether a call takes a workspace of so many bytes. Without its address it then ends as EINVAL, before
    anything is launched."""
    a = [P()] * 8 + [9, P(), 4, P(), hint, P(), batch, total, hq, hkv, d, 16, hq * d, hkv * d, hkv * d, 0.0, None,
                     ws_bytes, None, None]
    rc = code("mars_attn_chunk_q8", a)
    assert rc in (mars.EINVAL, mars.ENOSPACE)
    return rc == mars.EINVAL


def test_a_workspace_for_the_largest_call_is_enough_for_all():
    """Of no more sequences, rows and cached tokens, whatever forms the calls take; and what a call asks for grows
    with the hint, to 2 GB and some at most."""
    import random
    rng = random.Random(3)
    size = lambda *a: packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, *a)   # noqa: E731
    for i in range(4000):
        heads = rng.choice([(28, 4, 128), (4, 2, 64), (96, 1, 64), (16, 16, 128), (14, 2, 64), (130, 1, 64)])
        batch, total, hint = (int(2 ** rng.uniform(0, m)) for m in (9, 14, 20))
        most = size(batch, total, *heads, hint)
        assert most <= size(batch, total, *heads, hint + int(2 ** rng.uniform(0, 22)))
        assert most < (1 << 31) + (1 << 30)
        b, t, h = rng.randint(1, batch), rng.randint(1, total), rng.randint(0, hint)
        assert fits(batch, total, *heads, hint, most) and fits(b, t, *heads, h, most), (heads, batch, total, hint, b, t, h)
    # rows that take the few-row form in one batch and a larger tile in the next; pages beyond the limit
    for large, small in (((128, 256, 4096), (64, 256, 4096)), ((128, 23041, 16384), (128, 23041, 16385)),
                         ((12, 5532, 131072), (12, 5532, 2600)), ((12, 5532, 2600), (1, 5532, 2600))):
        args = lambda s: (s[0], s[1], 28, 4, 128, s[2])                                # noqa: E731
        assert fits(*args(small), size(*args(large)))
