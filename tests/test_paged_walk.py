"""The ragged prefill's schedule (PagedWalk, csrc/fa_paged.cuh) on the host: over random batches every CTA's
run as the header's own code finds it, with a warp's lanes emulated (paged_walk_host.cpp)."""
import collections
import os
import random
import subprocess

import pytest

from quantized_kv_cache_sm_gb300 import build as fa_build

HERE = os.path.dirname(os.path.abspath(__file__))
WHOLE, OVER = 8, 2  # PagedPlan::kWhole, kOver


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = tmp_path_factory.mktemp("paged_walk") / "walk"
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", fa_build.CSRC, "-o", str(exe),
                    os.path.join(HERE, "paged_walk_host.cpp")], check=True, capture_output=True)

    def run(new, lens, *, Hkv=2, causal=1, unit_tok=64, page=128, pps=None, rows=None, grid=152, first=0,
            starts=None):
        pps = pps or max(1, max(-(-n // page) for n in lens))
        starts = starts or [first + sum(new[:i]) for i in range(len(new) + 1)]
        args = [len(lens), Hkv, causal, unit_tok, 1000, page, pps, starts[-1] if rows is None else rows, grid,
                *starts, *lens]
        p = subprocess.run([str(exe)], input=" ".join(map(str, args)), text=True, capture_output=True)
        assert p.returncode == 0, (p.returncode, p.stderr)
        err, *rest = p.stdout.splitlines()
        return int(err), [tuple(map(int, x.split())) for x in rest]

    return run


def unit_blocks(new, lens, causal, unit_tok):
    """{(sequence, first token): 128-key blocks}: those that the unit's last token sees, at least one."""
    out = {}
    for b, (n, length) in enumerate(zip(new, lens)):
        for tok in range(0, n, unit_tok):
            keys = min(length, length - n + min(n, tok + unit_tok)) if causal else length
            out[b, tok] = max(1, -(-max(0, keys) // 128))
    return out


def check(segments, new, lens, Hkv, causal, unit_tok, grid):
    units = unit_blocks(new, lens, causal, unit_tok)
    pieces = collections.defaultdict(list)  # by unit
    runs = collections.defaultdict(list)    # by CTA
    for cta, b, tok, g, j0, j1, c_first, c_last, slot in segments:
        pieces[b, tok, g].append((cta, j0, j1, c_first, c_last, slot))
        runs[cta].append(((b, tok, g), j0, j1, c_first, c_last, slot))
    assert set(pieces) == {(b, tok, g) for b, tok in units for g in range(Hkv)}
    for (b, tok, g), ps in pieces.items():
        nb = units[b, tok]
        # the blocks once each, in CTA order, and all CTAs agree on who takes part and where
        assert [j for _, j0, j1, *_ in ps for j in range(j0, j1)] == list(range(nb))
        assert all(j1 > j0 for _, j0, j1, *_ in ps)
        assert len({p[3:] for p in ps}) == 1
        _, _, _, c_first, c_last, slot = ps[0]
        assert [p[0] for p in ps] == list(range(c_first, c_last + 1))
        assert nb > WHOLE or c_first == c_last
        assert slot in (0, 1)
    for cta, run in runs.items():
        assert 0 <= cta < grid
        taken = []
        for i, (unit, _, _, c_first, c_last, slot) in enumerate(run):
            # a unit that others began is the run's first, one that others go on with its last
            assert c_first == cta or i == 0
            assert c_last == cta or i == len(run) - 1
            if c_first != c_last:
                taken.append(slot if c_first == cta else 0)
        assert len(set(taken)) == len(taken), (cta, run)  # the CTA's pieces lie in different slots
        order = [(u[0], u[1], u[2]) for u, *_ in run]
        assert order == sorted(order)
    # an even cut: no run is longer than its share of the counts and half a whole unit at each end
    total = sum(Hkv * (OVER + nb) for nb in units.values())
    share = -(-total // min(grid, total)) if total else 0
    for run in runs.values():
        assert sum(j1 - j0 for _, j0, j1, *_ in run) <= share + OVER + WHOLE


def test_random_batches(walk):
    rng = random.Random(1)
    for _ in range(60):
        B = rng.choice([1, 2, 5, 31, 32, 33, 64, 70])
        top, ctx = rng.choice([(1, 9000), (6, 3000), (700, 700), (300, 20000), (40, 60)])
        new = [rng.choice([0, 1, rng.randrange(top + 1)]) for _ in range(B)]
        lens = [max(0, n + rng.choice([0, -3, rng.randrange(ctx)])) for n in new]
        kw = dict(Hkv=rng.choice([1, 2, 5, 8]), causal=rng.choice([0, 1, 1]),
                  unit_tok=rng.choice([2, 64, 256, 50]), grid=rng.choice([152, 148, 7, 1]))
        if kw["unit_tok"] == 2:
            new = [min(n, 60) for n in new]
        err, segments = walk(new, lens, first=rng.choice([0, 9]), page=rng.choice([16, 48, 128, 256]), **kw)
        assert err == 0
        check(segments, new, lens, **kw)


@pytest.mark.parametrize("Hkv,grid", [(1, 152), (8, 152), (8, 4)])
def test_edges_of_whole_and_cut_units(walk, Hkv, grid):
    """Units of 7 to 10 blocks, so that runs end on, just before and just after every count of them."""
    for n in range(1, 40):
        lens = [128 * (7 + (i + n) % 4) for i in range(n)]
        err, segments = walk([1] * n, lens, Hkv=Hkv, grid=grid)
        assert err == 0
        check(segments, [1] * n, lens, Hkv, 1, 64, grid)


def test_bad_batches(walk):
    """Starts out of order or range leave nothing to any CTA; a bad length is recorded and taken as the nearest
    good one."""
    for starts in ([0, 9, 4], [-1, 4, 13], [0, 4, 14], [5, 4, 13]):
        assert walk(None, [300, 200], starts=starts, rows=13) == (2, [])
    for n, taken in ((-1, 0), (-2 ** 31, 0), (385, 384), (2 ** 31 - 1, 384)):
        err, segments = walk([4, 9], [n, 200], pps=3)
        assert err == 2
        check(segments, [4, 9], [taken, 200], 2, 1, 64, 152)
    assert walk([0, 0], [300, 5]) == (0, [])
