"""Which tile and split the grouped products and adapters take (no GPU): the choices that grouped_choice.h
states with their times are the ones it makes, and options are kept."""
import os
import shutil
import subprocess

import pytest

from blackwell_tensor_core_02_gb300 import build

# rows, groups, N, K, of a product or (sums over rows) the matrices' gradient; tile and split, 0 a persistent grid
STATED = [("nt", 256, 1, 4096, 4096, 0, (128, 2)), ("nt", 512, 1, 2048, 2048, 0, (128, 2)), ("nt", 2000, 8, 2048, 2048, 0, (256, 0)),
          ("nt", 8192, 8, 1024, 1024, 0, (256, 0)), ("nt", 2, 64, 2048, 1024, 0, (16, 4)), ("nt", 4096, 64, 1024, 1024, 0, (128, 0)),
          ("tn", 8192, 1, 1024, 1024, 0, (128, 2)), ("tn", 3855, 1, 208, 208, 0, (64, 4)), ("tn", 8192, 8, 1024, 1024, 0, (256, 0)),
          ("tn", 6098, 10, 184, 88, 0, (64, 0)),
          ("lora", 64, 64, 4096, 4096, 16, (64, 4)), ("lora", 800, 8, 4096, 4096, 16, (256, 0)), ("lora", 2048, 32, 4096, 4096, 16, (128, 1)),
          ("lora", 256, 64, 1024, 1024, 32, (32, 2)), ("lora", 1, 1, 2048, 2048, 32, (16, 4))]

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "grouped_choice.h"

struct Sizes {
    int32_t groups, rows, I, J, R, rank;
};

int main(int argc, char **argv) {  // kind rows groups N K rank tile split, again and again
    for (int i = 1; i + 7 < argc; i += 8) {
        long v[7];
        for (int k = 0; k < 7; ++k) v[k] = std::atol(argv[i + 1 + k]);
        grouped_options o = {};
        o.tile = static_cast<int32_t>(v[5]), o.split = static_cast<int32_t>(v[6]);
        const bool sum = !std::strcmp(argv[i], "tn");
        const Sizes p = {int32_t(v[1]), int32_t(v[0]), int32_t(sum ? v[3] : v[2]), int32_t(sum ? v[2] : 0), int32_t(sum ? v[2] : v[3]), int32_t(v[4])};
        const linear_ops::Choice c = !std::strcmp(argv[i], "lora") ? linear_ops::choose_lora(p, 152, o)
                                                                   : linear_ops::choose(sum ? linear_ops::kGroupTN : linear_ops::kGroupNT, p, 152, o);
        std::printf("%d %d\n", c.tile, c.split);
    }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    where = tmp_path_factory.mktemp("choice")
    (where / "main.cpp").write_text(MAIN)
    exe = str(where / "main")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", build.INCLUDE, "-I", build.LINEAR_CSRC,
                    str(where / "main.cpp"), "-o", exe], check=True)

    def run(cases):
        args = [str(a) for case in cases for a in case]
        out = subprocess.run([exe, *args], check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, s.split())) for s in out.splitlines()]
    return run


def test_the_stated_choices(choose):
    got = choose([(*case[:6], 0, 0) for case in STATED])
    assert got == [case[6] for case in STATED]
    with open(os.path.join(build.LINEAR_CSRC, "grouped_choice.h")) as f:
        text = f.read()
    for stated in ("128 rows, 2 CTAs a tile: 13.5", "16, 4: 4.9", "64, 4: 6.9", "64 rows, 4 CTAs a tile: 16.8", "16, 4: 5.9"):
        assert stated in text


def test_options_are_kept(choose):
    """A tile or split that is asked for is taken (a split no longer than the sum), and with what goes with it."""
    cases, want = [], []
    for rows, groups, N, K in ((1, 1, 64, 64), (300, 7, 1000, 2048), (5000, 3, 8, 512)):
        for tile, split in ((16, 1), (32, 8), (128, 2), (256, -1), (64, -1)):
            cases.append(("nt", rows, groups, N, K, 0, tile, split))
            most = (K + 63) // 64
            while split > 1 and split > most:
                split //= 2
            want.append((tile, max(split, 0)))
    assert choose(cases) == want
    for tile, split in choose([("nt", 300, 7, 1000, 2048, 0, 0, s) for s in (1, 2, 4, 8)]):
        assert tile <= 128 and split > 0
    assert all(c == (256, 0) for c in choose([("lora", 300, 7, 1000, 2048, 16, t, s) for t, s in ((256, 0), (0, -1), (256, -1))]))
