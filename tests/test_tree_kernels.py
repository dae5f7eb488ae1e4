"""Which kernel the attention of drafted trees takes: the bounds that the GPU tests rely on give what they say."""
import os
import subprocess

import pytest

from kv8_tree_cases import KERNELS

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "w8a8_quantized_linear_channel_amd", "csrc")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "tree_plan_print")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}",
                    os.path.join(HERE, "native", "tree_plan_print.cpp"), "-o", exe], check=True)
    lines = [f"{c[2]} {c[3] // c[4]} {c[4]} {c[5]} {c[7]} {c[8]} {c[9]}\n" for c in KERNELS.values()]
    r = subprocess.run([exe], input="".join(lines), capture_output=True, text=True, timeout=60, check=True)
    return {name: tuple(map(int, line.split())) for name, line in zip(KERNELS, r.stdout.splitlines())}


@pytest.mark.parametrize("name", KERNELS)
def test_bounds_give_the_kernel(plans, name):
    per, splits, _ = plans[name]
    assert (per, splits > 1) == KERNELS[name][:2]


def test_every_kernel_is_among_them():
    # rows a workgroup x features x split, of those that there are (32 rows: 128 features only)
    want = {(16, d, s) for d in (64, 128, 256) for s in (False, True)} | {(32, 128, False), (32, 128, True)}
    want |= {(128 if d == 256 else 256, d, s) for d in (64, 128, 256) for s in (False, True)}
    assert {(c[0], c[5], c[1]) for c in KERNELS.values()} == want
