"""The rule that picks the 4-bit LM head's shape, asked on the host."""
import pytest

import device_text as D
import fp4_shapes as S

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "sv_lmhead_fp4_plan.h"
int main(int argc, char **argv)
{
    for (int i = 1; i + 1 < argc; i += 2) {
        const sv::Lm4Plan p = sv::lm4_plan(atoll(argv[i]), atoi(argv[i + 1]), 152);
        printf("%d %d %d %d %d %d\n", p.pair, p.H, p.RT, p.MT, p.NT, p.NB);
    }
}
"""


def _plans(tmp_path, sizes):
    out = D.run(MAIN, tmp_path, *[str(n) for s in sizes for n in s[:2]])
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_tested_sizes_reach_every_shape(tmp_path):
    for sizes, want in ((S.LONE, (0, 1)), (S.PAIR, (1, 1)), (S.TWO, (1, 2))):
        plans = _plans(tmp_path, sizes)
        assert [p[:2] for p in plans] == [want] * len(sizes)
    two = _plans(tmp_path, S.TWO)
    assert {p[2] % 2 for p in two} == {0, 1}                       # whole groups, and a last one of one row tile
    assert any(V % 8 for _, V, _ in S.TWO) and any(V % 8 == 0 for _, V, _ in S.TWO)
    # units of 76 pairs form more than one tile each somewhere
    assert any(p[3] * p[4] > 76 for p in two)
    assert [p[2] % 2 for p in _plans(tmp_path, S.ODD_LAST)] == [1] * len(S.ODD_LAST)


@pytest.mark.parametrize("M", [0, 1, 127, 128, 129, 256, 257, 300, 640, 1000, 2304, 40000, 1 << 20])
def test_plans_cover_the_product(M, tmp_path):
    sizes = [(M, V) for V in (1, 63, 64, 65, 500, 8191, 32003, 151936, 1 << 21)]
    for (_, V), (pair, H, RT, MT, NT, NB) in zip(sizes, _plans(tmp_path, sizes)):
        rows = 256 if pair else 128
        assert NB in (64, 128, 192) and (pair or H == 1) and H in (1, 2)
        assert RT * rows >= M > (RT - 1) * rows or (M == 0 and RT == 1)
        assert MT == -(-RT // H) and NT * NB >= V > (NT - 1) * NB
