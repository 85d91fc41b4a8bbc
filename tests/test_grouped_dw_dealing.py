"""Every tile of gemm_grouped_dw's output is computed by one workgroup (CPU):
the library's own plan and dealing, compiled for the host from its header and
walked tile by tile (tests/arith/grouped_dw_dealing.hip)."""
import os
import random
import subprocess

import pytest

from scaled_precision_gemm_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))

# wide outputs whose rows of tiles come in 16 parts or more, the last unit of rows of tiles not whole: (E, N, K, rows)
WIDE = [(1, 4608, 36864, 64), (1, 3584, 28672, 64), (1, 5376, 24576, 64), (1, 6400, 20480, 64), (1, 6656, 53248, 64),
        (2, 1792, 32768, 64), (3, 1280, 32768, 64), (1, 3328, 32768, 64), (1, 3328, 28672, 64), (5, 1280, 20480, 64),
        (2, 4320, 32768, 64), (3, 5472, 32768, 64), (1, 5120, 65536, 64), (1, 776, 262144, 64), (3, 520, 1 << 20, 64)]
# a tile and less, one expert's even units, parts of the experts' rows, most experts
OTHERS = [(1, 8, 8, 1), (1, 8, 8, 100000), (2, 8, 8, 0), (1, 512, 512, 32768), (1, 4096, 2048, 4000), (1, 2048, 2048, 4096),
          (8, 1024, 512, 8192), (64, 2048, 2048, 32768), (64, 2048, 1024, 29500), (1, 4096, 4096, 32768), (1, 8192, 8192, 8192),
          (1, 5120, 17408, 4096), (1, 34816, 5120, 4096), (16, 2048, 2048, 16384), (65536, 8, 16, 3000), (1000, 264, 520, 9)]


@pytest.fixture(scope="module")
def deal(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("dealing") / "grouped_dw_dealing")
    # (the device's part of the header is not compiled: nothing here runs on a GPU)
    r = subprocess.run([build.hipcc(), "--offload-host-only", "-O2", "-std=c++17", "-Wno-unused-command-line-argument",
                        "-I", build.CSRC, os.path.join(HERE, "arith", "grouped_dw_dealing.hip"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        r = subprocess.run([exe], input="".join("%d %d %d %d\n" % c for c in cases), capture_output=True, text=True)
        lines = r.stdout.splitlines()
        assert r.returncode == 0 and len(lines) == len(cases), r.stderr
        bad = [line for line in lines if " missing 0 twice 0 " not in line]
        assert not bad, "\n".join([f"{len(bad)} of {len(cases)}:"] + bad[:12])
        return [tuple(map(int, line.split("plan ")[1].split())) for line in lines]

    return run


@pytest.mark.parametrize("cases", [WIDE, OTHERS], ids=["wide", "others"])
def test_every_tile_once(deal, cases):
    deal(cases)


def test_every_tile_once_over_the_range(deal):
    rng, cases = random.Random(1), []
    while len(cases) < 3000:
        e = rng.choice([1, 1, 1, 2, 3, 5, 8, 60, 64, 128, 1000])
        n, k = 8 * int(2 ** rng.uniform(0, 12.5)), 8 * int(2 ** rng.uniform(0, 15))
        if rng.random() < 0.5:           # rows of tiles that split evenly
            k = -(-k // 2048) * 2048
        if e * (n // 128 + 1) * (k // 256 + 1) <= 100000:
            cases.append((e, n, k, int(2 ** rng.uniform(0, 17))))
    plans = deal(cases)
    # all kinds of plan are among them: rows in parts, units of one, two and four rows of tiles, whole and in parts
    assert {s > 1 for s, _, _ in plans} == {False, True} and {n for _, n, _ in plans} == {0, 1, 2}
    assert {k for _, n, k in plans if n} >= {0, 1, 2, 3}
