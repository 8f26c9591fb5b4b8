"""The counts behind the attention's plan, on the host: a program of the kernels' own header goes through lists in
order and lists out of order, and says how many numbers a plan of them stores and how many its scratch holds."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include "attn_internal.h"
#include <cstdio>
#include <vector>
using namespace hca;

// T group rows width, requests, offsets, groups, starts: what attn_api.hip and make_plan count of them
int main()
{
    int T, group, rows, width, B, G;
    while (std::scanf("%d %d %d %d %d", &T, &group, &rows, &width, &B) == 5) {
        std::vector<int> off(B + 1), starts;
        for (int& x : off)
            if (std::scanf("%d", &x) != 1)
                return 1;
        if (std::scanf("%d", &G) != 1)
            return 1;
        starts.resize(G + 1);
        for (int& x : starts)
            if (std::scanf("%d", &x) != 1)
                return 1;
        const int64_t room = 2 * (int64_t(T) * group / rows) + B + G;
        int64_t tiles = 0;
        for (int s = 0; s < B + G; ++s) {
            int lo, hi, r0 = s, r1 = s + 1;
            if (s >= B)
                clamped_range(B, starts.data(), s - B, s - B + 1, r0, r1);
            clamped_range(T, off.data(), r0, r1, lo, hi);
            if (lo < 0 || hi < lo || hi > T)
                return 2;
            tiles += tiles_of(hi - lo, group, rows);
        }
        const int64_t stored = planned((int)tiles, (int)room) ? tiles : 0;
        const Scratch at = scratch_of(T, group, rows, width, B + G, room, true);
        std::printf("%lld %lld %lld %lld\n", (long long)room, (long long)tiles, (long long)(4 * plan_numbers(B + G, stored)),
                    (long long)(at.ranges - at.plan));
    }
}
"""


@pytest.fixture(scope="module")
def counted(tmp_path_factory):
    from hyper_connection_residual_amd import build
    here = tmp_path_factory.mktemp("plan")
    source, program = here / "plan.hip", here / "plan"
    source.write_text(PROGRAM)
    flags = [f for f in build.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([build.hipcc(), *flags, "-I", build.ATTN_CSRC, "-I", build.PROJ_CSRC, "-I", build.INCLUDE, str(source), "-o", str(program)],
                   check=True, capture_output=True, text=True)

    def run(calls):
        lines = "\n".join(" ".join(map(str, [T, group, rows, width, len(off) - 1, *off, len(starts) - 1, *starts])) for T, group, rows, width, off, starts in calls)
        out = subprocess.run([str(program)], input=lines, check=True, capture_output=True, text=True).stdout.splitlines()
        assert len(out) == len(calls)
        return [tuple(map(int, x.split())) for x in out]

    return run


def test_lists_in_order_have_the_tiles_that_the_scratch_has_room_for(counted):
    rng, calls = random.Random(1), []
    for _ in range(2000):
        B, group, T = rng.choice([1, 3, 64, 65, 500, 2048]), rng.choice([1, 3, 5, 8]), rng.randint(1, 4000)
        G = rng.choice([1, 2, 9, 70])
        off = sorted(rng.randint(0, T) for _ in range(B + 1))
        starts = sorted(rng.randint(0, B) for _ in range(G + 1))
        calls.append((T, group, 128, 64, off, starts))
    for room, tiles, stored, bytes_ in counted(calls):
        assert tiles <= room and stored <= bytes_


def test_lists_out_of_order_store_no_more_than_the_scratch_holds(counted):
    """Every second request, or every second prefix, has all tokens: far more tiles than lists in order have."""
    rng, calls = random.Random(2), []
    for T, group, B in ((512, 5, 64), (8192, 5, 256), (4096, 1, 1000), (4000, 8, 2048)):
        calls.append((T, group, 128, 64, [0, T] * (B // 2) + [0], [0, B]))
        calls.append((T, group, 128, 64, [T * b // B for b in range(B + 1)], [0, B] * 200 + [0]))
    assert all(tiles > room for room, tiles, _, _ in counted(calls))
    for _ in range(2000):
        B, group, T, G = rng.choice([1, 3, 64, 65, 500, 2048]), rng.choice([1, 3, 5, 8]), rng.randint(1, 4000), rng.choice([1, 2, 9, 70, 500])
        wild = lambda top: rng.choice([rng.randint(0, top), rng.randint(0, top), 0, top, -2 ** 31, 2 ** 31 - 1])  # noqa: E731
        calls.append((T, group, 128, 64, [wild(T) for _ in range(B + 1)], [wild(B) for _ in range(G + 1)]))
    for room, tiles, stored, bytes_ in counted(calls):
        assert stored <= bytes_
