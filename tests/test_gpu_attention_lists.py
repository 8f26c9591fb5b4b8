"""The attention's scratch and outputs between guards, whatever the lists on the device hold: lists in order with
ranges of every token's own, and lists out of order, which a plan may not follow past its room."""
import random

import pytest
import torch

from test_gpu_attention import BF, Call, a, case, guarded, ints, ranges  # noqa: F401 (a: the fixture)

pytestmark = pytest.mark.gpu


def run_guarded(a, c, offsets=None, lengths=None, starts=None, prefix_lengths=None, first=None, last=None, slopes=None):
    """(results, whether what lies around the scratch and the results is as it was) of a call with these lists."""
    lib, T = a.library(), c.T
    B = len(c.requests)
    batch = a.Batch(c.offsets if offsets is None else offsets, c.lengths if lengths is None else lengths, c.table)
    shared = None
    if c.prefixes:
        groups = len(c.prefixes) if starts is None else len(starts) - 1
        table = c.prefix_table if starts is None else c.prefix_table[torch.arange(groups, device="cuda") % len(c.prefixes)].contiguous()
        lens = ints(c.prefixes if starts is None else [c.prefixes[g % len(c.prefixes)] for g in range(groups)]) if prefix_lengths is None else prefix_lengths
        shared = a.SharedPrefix(ints(c.starts) if starts is None else ints(starts), lens, table)
    size = lib.hc_attend_work(T, c.Hq, c.Hkv, c.D, B, shared.groups if shared else 0)
    assert size > 0
    work, work_kept = guarded(size)
    out, out_kept = guarded(2 * c.q.numel())
    point = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    rest = (c.scale, 0.0, point(slopes), point(first), point(last), out.data_ptr(), c.Hq * c.D, c.D, work.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    if shared:
        status = lib.hc_attend_shared(T, c.Hq, c.q.data_ptr(), c.Hq * c.D, c.D, c.cache._at, batch._at, shared._at, *rest)
    else:
        status = lib.hc_attend(T, c.Hq, c.q.data_ptr(), c.Hq * c.D, c.D, c.cache._at, batch._at, *rest)
    assert status == a.HC_OK
    torch.cuda.synchronize()
    return out.view(c.dtype).view(c.q.shape), work_kept() and out_kept()


# (requests, their new tokens, prefixes, query heads, cache heads, columns)
WILD = [
    (64, 8, [300], 10, 2, 64),       # tiles of 128 rows, 65 segments
    (256, 6, [400, 70], 5, 1, 128),
    (9, 200, [200], 8, 2, 256),
    (1000, 4, [90], 2, 2, 64),
    (2048, 1, [33] * 5, 4, 1, 64),
    (2048, 2, [], 2, 2, 64),         # tiles of 16 rows
    (100, 8, [], 1, 1, 128),
    (300, 20, [], 2, 1, 256),        # of 32
    (40, 300, [], 4, 1, 64),         # of 128
    (12, 900, [], 4, 4, 128),        # of 256
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("layout", range(len(WILD)))
def test_lists_out_of_order_stay_inside_scratch_and_output(a, layout, masked):
    """Offsets and prefixes' starts that give all tokens to every second request or prefix, and any numbers.  Nothing but
    scratch and output is written; what lists in order give is right afterwards."""
    B, n, prefixes, Hq, Hkv, D = WILD[layout]
    case("wild lists", layout, masked)
    rng = random.Random(layout)
    starts = [B * g // len(prefixes) for g in range(len(prefixes) + 1)] if prefixes else None
    c = Call(a, [(n, n + 1 + b % 60) for b in range(B)], Hq, Hkv, D, 16, BF, seed=40 + layout, prefixes=prefixes, starts=starts)
    T = c.T
    first, last = ranges(c, "any") if masked else (None, None)
    wild = lambda top: rng.choice([rng.randint(0, top), rng.randint(0, top), 0, top, -2 ** 31, 2 ** 31 - 1])  # noqa: E731
    of_all = lambda top, k: ([0, top] * k)[:k]  # noqa: E731
    for i, off in enumerate([of_all(T, B + 1), of_all(T, B + 2)[1:], [wild(T) for _ in range(B + 1)], c.off[::-1], None, None, None]):
        there = None
        if prefixes:
            there = [None, None, [wild(B) for _ in range(200)], starts[::-1], of_all(B, 401), [wild(B) for _ in range(500)], of_all(B, 2049)][i]
        print("lists", i, flush=True)
        _, kept = run_guarded(a, c, None if off is None else ints(off), starts=there, first=first, last=last)
        assert kept, i
    got, kept = run_guarded(a, c, first=first, last=last)
    assert kept
    c.check(got, c.want(first=first, last=last))
