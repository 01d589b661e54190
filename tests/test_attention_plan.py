"""The deal of attention's tiles to workgroups (no GPU): every tile of every
unit exactly once, parts in places of their own that the join finds."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "attn_plan")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "bit_svdquant_diffusion_amd", "csrc"),
                    os.path.join(ROOT, "tests", "attn_plan.cpp"), "-o", exe], check=True)

    def run(cases):
        text = "".join(" ".join(str(int(v)) for v in c) + "\n" for c in cases)
        r = subprocess.run([exe], input=text, stdout=subprocess.PIPE, text=True, timeout=300)
        assert r.returncode == 0
        return r.stdout.splitlines()
    return run


def _cases(queries, keys, group, causal, heads):
    rows = queries * group
    return [(rows, keys, group, keys - queries, causal, 0, heads, block) for block in (128, 256)] + \
        [(keys, rows, group, keys - queries, causal, 1, heads, block) for block in (128, 256)]


def test_every_tile_once(plan):
    rng = random.Random(5)
    cases = []
    for queries, keys, group, heads in [(4608, 4608, 1, 24), (1, 65536, 4, 8), (1531, 1601, 3, 8), (4096, 77, 1, 40), (1, 1, 1, 1),
                                        (5, 0, 1, 2), (0, 5, 1, 2), (1 << 20, 1 << 20, 1, 1), (100, 30, 2, 3), (256, 256, 1, 256),
                                        (300, 100000, 64, 1), (8192, 64, 1, 31), (16384, 16384, 1, 13)]:
        for causal in (0, 1):
            cases += _cases(queries, keys, group, causal, heads)
    for _ in range(400):
        group = rng.choice([1, 1, 2, 3, 8])
        heads = int(2 ** rng.uniform(0, 9))
        cases += _cases(int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 14)), group, rng.random() < 0.5, heads)
    got = plan(cases)
    assert len(got) == len(cases)
    bad = [g for g in got if not g.startswith("ok")]
    assert not bad, bad[:5]
    assert any(g.split()[2] != "0" for g in got) and any(g.split()[2] == "0" for g in got)


def test_few_units_are_cut_and_many_are_not(plan):
    rows = lambda *a: _cases(*a)[1]   # noqa: E731 (blocks of 256)
    got = plan([rows(4608, 4608, 1, 0, 24), rows(1, 65536, 4, 0, 8), rows(256, 65536, 1, 0, 250), _cases(4096, 77, 1, 0, 40)[2],
                rows(1, 65536, 4, 0, 1)])
    assert got == ["ok 432 0", "ok 256 32", "ok 250 0", "ok 240 11", "ok 256 4"]
