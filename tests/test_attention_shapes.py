"""The shapes of attention's launches (no GPU): every size gets one that a
kernel exists for, and every kind of launch has sizes."""
import os
import random
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_size_has_a_launch(tmp_path):
    exe = str(tmp_path / "attn_shapes")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "bit_svdquant_diffusion_amd", "csrc"),
                    os.path.join(ROOT, "tests", "attn_shapes.cpp"), "-o", exe], check=True)
    rng, lines = random.Random(3), []
    size = lambda most: int(2 ** rng.uniform(0, most))   # noqa: E731
    for _ in range(20000):
        kv = size(5)
        lines.append((size(6), size(13) - (rng.random() < 0.02), size(16), kv * size(5), kv, 8 * rng.randint(1, 16), rng.randint(0, 1),
                      rng.randint(0, 1)))
    r = subprocess.run([exe], input="".join(" ".join(map(str, c)) + "\n" for c in lines), stdout=subprocess.PIPE, text=True,
                       timeout=300)
    got = r.stdout.splitlines()
    assert r.returncode == 0 and len(got) == len(lines)
    bad = [g for g in got if not g.startswith("ok")]
    assert not bad, bad[:5]
    assert {g.split()[1] for g in got} == {"8/1/0", "8/1/1", "4/2/0", "4/2/1", "4/1/0"}
    assert {g.split()[2] for g in got} == {"8/1/0", "8/1/1", "4/2/0", "4/2/1", "4/1/0"}
