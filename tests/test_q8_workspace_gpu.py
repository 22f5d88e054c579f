"""Attention over the 8-bit cache on workspaces of other sizes than a call's own (needs a GB300)."""
import pytest
import torch

from block_masked_token_gb300 import mars, packed
from packed_util import cuda
from test_q8_calls import fits
from test_q8_gpu import check_chunk8, hint_of, make8, run_chunk8, same

pytestmark = pytest.mark.gpu

HEADS = (28, 4, 128)


def size(batch, total, hint):
    return packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, batch, total, *HEADS, hint)


def test_many_rows_with_less_room_for_pages():
    """From no room for unpacked pages to room for all: what has none is computed from the codes."""
    x = make8([700, 1, 800, 40], *HEADS, [500, 900, 20, 3000], seed=900)
    y, args = cuda(x), (4, 1541, 3100)
    full = size(*args)
    low, high = 0, full                              # the least that the call takes
    while low < high:
        mid = (low + high) // 2
        if fits(4, 1541, *HEADS, 3100, mid):
            high = mid
        else:
            low = mid + 1
    assert low < full - (1 << 20)
    page = 4 * 4 * 16 * 128 * 4
    for bytes_ in (low, low + page // 2, low + (full - low) // 40, low + (full - low) // 5, full - page, full, full + 999):
        ws = torch.full((bytes_,), 0xa5, dtype=torch.uint8, device="cuda")
        guarded = torch.full((bytes_ + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
        o, st = run_chunk8(y, hint=3100, ws=guarded[:bytes_])
        assert st == 0 and (guarded[bytes_:] == 0xa5).all()
        check_chunk8(x, o, rows=[0, 39, 600, 699, 799])
        again, _ = run_chunk8(y, hint=3100, ws=ws)
        assert same(o, again)
    with pytest.raises(mars.MarsError):
        run_chunk8(y, hint=3100, ws=ws[:low - 1])


def test_smaller_calls_on_the_largest_calls_workspace():
    ws = torch.full((size(40, 2000, 5000),), 0xa5, dtype=torch.uint8, device="cuda")
    for seed, (lens, old) in enumerate([([1] * 40, [100 * i for i in range(40)]), ([16] * 40, [100 * i for i in range(40)]),
                                        ([1800, 1], [300, 4000]), ([200], [0]), ([3], [4900]), ([50] * 40, [7 * i for i in range(40)])]):
        x = make8(lens, *HEADS, old, seed=910 + seed)
        for hint in (hint_of(x), 5000):
            o, st = run_chunk8(cuda(x), hint=hint, ws=ws)
            assert st == 0
            check_chunk8(x, o, rows=[0, 15, 49, 199, 1799])


@pytest.mark.parametrize("lens, old, hint", [([3, 1], [200, 5], 5000), ([16] * 30, [300] * 30, 900),
                                             ([1400, 3], [300, 40], 1800)], ids=["few", "middle", "many"])
def test_the_bindings_refuse_a_workspace_that_is_too_small(lens, old, hint):
    x = make8(lens, *HEADS, old, seed=920)
    y = cuda(x)
    assert size(len(lens), sum(lens), hint) > 16
    for ws in (torch.empty(16, dtype=torch.uint8, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")):
        with pytest.raises(mars.MarsError):
            run_chunk8(y, hint=hint, ws=ws)
        with pytest.raises(mars.MarsError):
            run_chunk8(y, hint=hint, ws=ws, stream=torch.cuda.current_stream())


def test_more_tiles_than_ctas_make_ready():
    """Own rows and pages of more than 3,100 groups of 16, which 16 CTAs per SM take in turn."""
    lens, old = [190 + i for i in range(12)], [4000 + 13 * i for i in range(12)]
    x = make8(lens, *HEADS, old, seed=930)
    y = cuda(x)
    for hint in (hint_of(x), 131072):
        o, st = run_chunk8(y, hint=hint)
        assert st == 0
        check_chunk8(x, o, rows=[0, 17, 100, 189])
