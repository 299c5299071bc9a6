"""The product's choice between single waves and tiles (choice.h) where both were
measured and one is the faster by a sixth or more, with even runs or, where
they are uneven, by more than that."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "matrix_optimizer_amd", "csrc")

# (rows, experts, n, whole 16-byte rows, bf16 results, waves)
MEASURED = [
    (96, 64, 4096, True, True, True),         # a served batch, 276 us
    (512, 64, 4096, True, True, False),       # all with one expert 288 and 81, eight with each 398 and 375
    (1024, 64, 4096, True, True, False),      # 468 and 377
    (1, 1, 4096, True, True, True),           # 9 and 49
    (64, 1, 4096, True, True, True),          # 22 and 53
    (64, 1, 8192, True, True, True),          # 155 and 203 with k of 28672
    (16, 1, 8192, True, True, True),          # 62 and 189
    (64, 1, 28672, True, True, False),        # 153 and 64
    (64, 4, 4096, True, True, True),          # 31 and 53
    (256, 8, 4096, True, True, False),        # 101 and 57
    (64, 1, 4096, True, False, True),         # 22 and 107
    (8192, 128, 2048, True, False, False),    # 794 and 401; half of them with one expert 1236 and 475
    (4096, 64, 4096, True, False, False),     # 1172 and 686; all with one expert 1165 and 298
    (64, 64, 4096, True, False, True),        # 464 and 663
    (256, 8, 4096, True, False, False),       # 109 and 71
    (128, 2, 8192, True, False, True),        # 85 and 120
    (32, 1, 28672, True, False, True),        # 110 and 132
    (32, 8, 4096, True, False, True),         # 52 and 67
    (16384, 256, 512, True, False, False),    # 220 and 111; all with one expert 1270 and 56
    (4096, 64, 2048, False, True, False),     # 458 and 121
    (256, 64, 2048, False, True, False),      # 154 and 111
    (32, 2, 2048, False, True, True),         # 16 and 60
    (512, 16, 1371, False, False, False),     # 92 and 48
    (16, 8, 2048, False, False, True),        # 50 and 83
    (128, 8, 2048, False, False, True),       # 67 and 85
    (128, 2, 4096, False, False, True),       # 71 and 84
    (64, 1, 28672, False, True, False),       # 392 and 136
]


@pytest.fixture(scope="module")
def limit(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    src, exe = d / "choice.cpp", d / "choice"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include "choice.h"\nint main(int, char** v) {\n'
                   '  std::printf("%lld\\n", (long long)muon::most_rows_of_waves(std::atoll(v[1]), *v[2] == 49, *v[3] == 49));\n}\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return lambda tiles, large, pieces: int(subprocess.run([str(exe), str(tiles), str(int(large)), str(int(pieces))],
                                                           capture_output=True, text=True, check=True).stdout)


@pytest.mark.parametrize("rows,experts,n,pieces,bf16,waves", MEASURED)
def test_measured_sizes_take_the_faster_kernel(limit, rows, experts, n, pieces, bf16, waves):
    large = bf16 and pieces
    tiles = min(experts, rows) * -(-n // (256 if large else 128))
    assert (rows <= limit(tiles, large, pieces) * experts) == waves


def test_limits(limit):
    for large, pieces in ((True, True), (False, True), (False, False)):
        got = [limit(t, large, pieces) for t in (0, 1, 16, 64, 128, 256, 1024, 1 << 20, 1 << 31)]
        assert got == sorted(got, reverse=True) and got[0] == 64 and got[-1] >= 1
