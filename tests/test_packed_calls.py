"""The C form of packed.py's calls (csrc/packed_calls.c): the arguments that reach the library,
and what it declines, with host tensors that say they are on the GPU and entry points that
record their arguments."""
import ctypes
import glob
import os

import pytest
import torch

from block_masked_token_gb300 import mars, packed

NAMES = ("mars_attn_packed", "mars_attn_packed_grad", "mars_attn_chunk", "mars_kv_append")
STREAM = 77


class Host:
    def __init__(self, t, device=0):
        self.t, self.device_index = t, device

    def __getattr__(self, n):
        return getattr(self.t, n)

    def get_device(self):
        return self.device_index


@pytest.fixture()
def calls():
    """The module set up with recorders: (module, list of the arguments of the calls made)."""
    if not os.path.exists(mars._LIB_PATH) or not glob.glob(
            os.path.join(os.path.dirname(packed.__file__), "_packed_calls*.so")):
        from block_masked_token_gb300.build import build_library
        build_library()
    from block_masked_token_gb300 import _packed_calls
    made, keep = [], []

    def recorder(name):
        argtypes = getattr(mars.lib(), name).argtypes

        def record(*a):
            made.append(a)
            return 5
        keep.append(ctypes.CFUNCTYPE(ctypes.c_int, *argtypes)(record))
        return ctypes.cast(keep[-1], ctypes.c_void_p).value

    _packed_calls.setup(Host, torch.bfloat16, torch.int32, torch.float32, torch.uint8, lambda: 0,
                        lambda dev: STREAM + dev, *map(recorder, NAMES))
    yield _packed_calls, made
    packed._calls = None                  # set up afresh where it is used next


def bf(*shape):
    return Host(torch.zeros(*shape, dtype=torch.bfloat16))


def i32(*shape):
    return Host(torch.zeros(*shape, dtype=torch.int32))


def arguments(name):
    """Positional arguments of the C form, and what the library has to get."""
    total, hq, hkv, d, batch, pages, width = 7, 4, 2, 64, 3, 9, 5
    qkv = torch.zeros(total, hq + 2 * hkv, d, dtype=torch.bfloat16)
    q, k, v = (Host(t) for t in qkv.split([hq, hkv, hkv], dim=1))
    dqkv = torch.zeros(total, 10, d, dtype=torch.bfloat16)
    dq, dk, dv = Host(dqkv[:, :hq]), Host(dqkv[:, hq:hq + hkv]), bf(total, hkv, d)
    o, do, lse = bf(total, hq, d), bf(total, hq, d), Host(torch.zeros(hq, total))
    cu, lens, new, slots = i32(batch + 1), i32(batch), i32(batch), i32(total)
    table, status = i32(batch, width), i32(1)
    kp, vp = bf(pages, hkv, 16, d), bf(pages, hkv, 16, d)
    ws = Host(torch.zeros(300, dtype=torch.uint8))
    p = lambda *ts: tuple(t.data_ptr() for t in ts)                  # noqa: E731
    wide = (hq + 2 * hkv) * d
    if name == "attn_packed":
        return ([q, k, v, cu, o, ws, lse, 0.25, status],
                (*p(q, k, v, cu, o, lse), batch, total, hq, hkv, d, wide, wide, wide, 0.25, *p(ws),
                 300, *p(status), STREAM))
    if name == "attn_packed_grad":
        return ([q, k, v, o, do, lse, cu, dq, dk, dv, ws, 0.5, None],
                (*p(q, k, v, o, do, lse, cu, dq, dk, dv), batch, total, hq, hkv, d, wide, wide,
                 wide, 640, 640, hkv * d, 0.5, *p(ws), 300, None, STREAM))
    if name == "attn_chunk":
        return ([q, k, v, cu, kp, vp, table, lens, 99, o, ws, status, 0.0, 16],
                (*p(q, k, v, cu, kp, vp), pages, *p(table), width, *p(lens), 99, *p(o), batch,
                 total, hq, hkv, d, 16, wide, wide, wide, 0.0, *p(ws), 300, *p(status), STREAM))
    return ([k, v, cu, kp, vp, table, lens, new, slots, status, 16],
            (*p(k, v, cu, lens, new, table), width, *p(kp, vp), pages, *p(slots), batch, total, hkv,
             d, 16, wide, wide, *p(status), STREAM))


@pytest.mark.parametrize("name", [n[5:] for n in NAMES])
def test_arguments_reach_the_library(calls, name):
    module, made = calls
    given, want = arguments(name)
    assert getattr(module, name)(*given) == 5
    assert made == [want]


@pytest.mark.parametrize("name", [n[5:] for n in NAMES])
def test_every_wrong_argument_is_declined(calls, name):
    """Each tensor in turn: of another type, shape, device or layout, or no tensor at all."""
    module, made = calls
    call = getattr(module, name)
    given, _ = arguments(name)
    for i, x in enumerate(given):
        bad = [object(), "x"]
        if isinstance(x, Host):
            t = x.t
            bad += [Host(t.to(torch.float64)), Host(t, device=1), Host(t, device=-1), Host(t[None]),
                    Host(torch.zeros(*(s + 1 for s in t.shape), dtype=t.dtype))
                    if t.dtype != torch.uint8 else Host(t.to(torch.int8)),
                    Host(torch.zeros(*(2 * s for s in t.shape), dtype=t.dtype)[
                        tuple(slice(0, None, 2) for _ in t.shape)])]
            if t.dim() == 1 and t.shape[0] == 1:
                bad.pop()                 # one element has no stride to be wrong
            if t.dim() == 1 and t.shape[0] == 4 and name.startswith("attn_packed"):
                del bad[-2]               # more boundaries are more sequences
        elif isinstance(x, float):
            bad.append(None)
        elif isinstance(x, int) and x == 99:
            bad += [-1, 1 << 31, 1 << 70, 9.0]
        for y in bad:
            assert call(*given[:i], y, *given[i + 1:]) is None, (i, y)
        if x is not None and i < len(given) - 1 and not (isinstance(x, Host) and name in (
                "attn_packed", "kv_append", "attn_chunk") and x in given[6:]):
            assert call(*given[:i], None, *given[i + 1:]) is None, i
    assert not made
    assert call(*given[:-1]) is None and call() is None
    if name in ("attn_chunk", "kv_append"):
        assert all(call(*given[:-1], page) is None for page in (0, -1, 1 << 31, 32, "x"))
    assert not made


def test_rows_of_odd_layouts(calls):
    module, made = calls
    given, _ = arguments("kv_append")
    k = given[0].t
    for t, pitch in ((torch.zeros(7, 2, 64, dtype=k.dtype), 128), (k, k.stride(0)),
                     (torch.zeros(7, 3 * 64 + 8, dtype=k.dtype)[:, :128].view(7, 2, 64), 200)):
        assert module.kv_append(Host(t), *given[1:]) == 5
        assert made[-1][16] == pitch
    for t in (torch.zeros(7, 64, 2, dtype=k.dtype).transpose(1, 2),
              torch.zeros(1, 2, 64, dtype=k.dtype).expand(7, 2, 64),
              torch.zeros(7, 2 * 64 + 4, dtype=k.dtype)[:, :128].view(7, 2, 64)):
        assert module.kv_append(Host(t), *given[1:]) is None
