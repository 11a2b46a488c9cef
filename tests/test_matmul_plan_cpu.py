"""How 8-bit products are taken (qg_matmul_plan.h), by sizes and CUs, on the host."""
import math
import random

import pytest

from matmul_plan_util import REACHED, SQUARE, plan, plans

ROWS = [256, 192, 128, 64, 128]
COLS = [256, 256, 256, 256, 128]        # of W


@pytest.mark.parametrize("kind,cut,head,S,I,O,gated", REACHED)
def test_sizes_reach_what_they_are_tested_for(kind, cut, head, S, I, O, gated):
    p = plan(S, I, O, gated=gated)
    assert p.tile and p.kind == kind and (p.parts > 1) == cut
    assert (p.head_kind if p.head else None) == head


def test_every_way_but_the_rarest_is_among_them():
    """All kinds in one launch, whole and in parts, plain and gated; and behind a first
    launch all but 256 rows, which come there only in parts of very long K."""
    def some(kind, cut, head):
        return {g for k, c, h, *_, g in REACHED
                if (k, c, h is not None) == (kind, cut, head)}
    for kind in range(5):
        assert some(kind, False, False) == some(kind, True, False) == {False, True}
    for kind in range(1, 5):
        assert some(kind, False, True) == {False, True}


def test_parts_heads_and_kinds_are_sound():
    r = random.Random(5)

    def size(lo, hi):
        return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))
    qs = []
    for _ in range(20000):
        gated = r.random() < 0.5
        qs.append((size(1, 1 << 24), r.choice([0, 0, 0, size(1, 1024)]), size(1, 1 << 20),
                   2 * size(1, 1 << 20), r.random() < 0.7, gated, r.random() < 0.7,
                   r.random() < 0.9, r.choice([256, 256, 80, 8])))
    for q, p in zip(qs, plans(qs)):
        R, E, I, O, bf16, gated, direct, fits, ncu = q
        oc, steps = (O // 2 if gated else O), -(-I // 128)
        if not p.tile:
            assert p.parts == 1 and p.bm in (16, 32, 64), q
            assert not fits or (R <= 64 if not E else R <= 16), q
            continue
        assert fits and p.bm == ROWS[p.kind], q
        if not (bf16 and direct):
            assert p.kind == SQUARE and p.head == 0, q
        if E:                            # the kinds that have grouped kernels
            assert (p.parts, p.head) == (1, 0) and R > 16, q
            assert p.kind in ((0, 2) if bf16 and direct else (SQUARE,)), q
        if p.parts > 1:                  # every part has steps; a tile for every slot at most
            per = -(-(-(-steps // p.parts)) // 4) * 4
            assert (p.parts - 1) * per < steps <= p.parts * per, q
            rest = oc - p.head
            tiles = -(-R // ROWS[p.kind]) * -(-rest // (COLS[p.kind] // (2 if gated else 1)))
            assert tiles * p.parts <= ncu * (2 if p.kind == SQUARE else 1) and R <= 4096, q
        if p.head:                       # whole tiles, and some columns behind them
            assert 0 < p.head < oc and p.head % (COLS[p.head_kind] // (2 if gated else 1)) == 0, q


def test_by_hand():
    # up to 16 rows of weights below 64 MB stream; grouped ones up to 16 rows in all
    assert not plan(16, 4096, 4096).tile and plan(16, 16384, 7168).tile
    assert not plan(16, 7168, 2048, E=256).tile and plan(17, 7168, 2048, E=256).tile
    assert plan(4096 * 8, 7168, 2048, E=256).kind == 2
    assert plan(4096 * 8, 7168, 2048, E=64).kind == 0
    # rows off 16 bytes and f32 take tiles of 128 x 128, K steps and all
    assert plan(300, 1024, 768, direct=False).kind == SQUARE
    assert plan(300, 1024, 768, bf16=False).kind == SQUARE
    # offsets beyond 32 bits stream
    assert not plan(300, 1024, 768, fits=False).tile
