"""The grouped-head work partition, walked on the host (gqa_partition.cu includes the kernels' own header): every item
and every key tile belongs to exactly one CTA, in order, at sizes that no GPU run reaches too."""
import os
import subprocess

import pytest

from long_context_sparse_10_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("partition") / "gqa_partition")
    subprocess.run([build._nvcc(), *build.ARCH, "-O2", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", exe,
                    os.path.join(HERE, "gqa_partition.cu")], check=True, capture_output=True)

    def run(op, Hkv, G, n, lens, ctas=148):
        """Units of the list, with the tiles the calls choose for chunks of up to max(n) tokens."""
        tpt = min(128 // G, max(n))
        tpb = tpt * (2 if op == "attention" and max(n) * G > 128 else 1)
        args = [str(x) for pair in zip(n, lens) for x in pair]
        r = subprocess.run([exe, op, str(Hkv), str(G), str(tpt), str(tpb), str(ctas), *args], capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return int(r.stdout)

    return run


BATCHES = [
    ([1], [1]), ([1] * 300, [100] * 300), ([2048, 513, 1, 777, 0, 4000, 31], [2048, 513, 1, 777, 0, 4000, 31]),
    ([0, 9, 300, 0], [0, 9, 400, 500]), ([5, 130, 4], [3, 200, 0]), ([512, 300, 77], [16384, 5001, 700]),
    ([1] * 8, [131072] * 8),
]


@pytest.mark.parametrize("op", ["attention", "weight"])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (8, 4), (3, 50), (1, 128)])
@pytest.mark.parametrize("n,lens", BATCHES)
def test_ordinary_batches(walk, op, Hkv, G, n, lens):
    for ctas in (1, 7, 148):
        assert walk(op, Hkv, G, n, lens, ctas) >= 0


@pytest.mark.parametrize("op,Hkv,G,n,L,units", [
    # one head of one sequence counts 2^32 units and more
    ("attention", 1, 128, 1_500_000, 1_500_000, 1 << 32),
    ("attention", 2, 128, 1_500_000, 1_500_000, 1 << 33),
    ("attention", 1, 64, 2_100_000, 2_100_000, 1 << 32),
    ("weight", 1, 128, 1_500_000, 1_500_000, 1 << 32),
    ("weight", 3, 100, 1_500_000, 1_500_000, 1 << 32),
    # one CTA's share counts 2^31 units and more
    ("attention", 1, 1, 300_000_000, 300_000_000, 148 << 31),
    ("attention", 1, 16, 40_000_000, 40_000_000, 148 << 31),
    ("weight", 1, 1, 300_000_000, 300_000_000, 148 << 31),
])
def test_counts_beyond_32_bits(walk, op, Hkv, G, n, L, units):
    assert walk(op, Hkv, G, [n], [L]) >= units
    assert walk(op, Hkv, G, [5, n, 700], [300, L, 700]) >= units
