"""The cut of the launches over the paged cache, checked on the host over the admitted sizes."""
import os
import subprocess

import pytest

from w8a8_quantized_linear_channel_amd import _lib as E

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "w8a8_quantized_linear_channel_amd", "csrc")


def test_every_launch_is_within_its_limits(tmp_path):
    exe = str(tmp_path / "kv_plan_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}",
                    os.path.join(HERE, "native", "kv_plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.skipif(not os.path.exists(E.LIB_PATH), reason="libq8.so not built")
def test_rows_past_32_bits_are_refused():
    """Tokens x heads that share a kv head are a 32-bit count in the kernels (fake pointers, never dereferenced)."""
    P, L = 0x10000, E.lib()
    for T, Hq, want in ((1 << 26, 32, 2), (1 << 30, 2, 2), ((1 << 26) - 64, 32, None)):
        r = L.q8_attention_kv8(P, Hq * 64, E.Q8_BF16, T, Hq, 1, 64, P, P, P, 1, 10, 4, 64, P, P, P, P, 50, 64, 0.1, 1, -1, P,
                               None, P, 1 << 40, None)
        assert r == (want or E.Q8_ERR_BAD_ARG), (T, Hq)      # past the sizes: the window of -1 is refused next
        assert (L.q8_attention_workspace_bytes(T, Hq, 1, 64, 1, 1, 100000, 0) == 0) == (want is not None)
