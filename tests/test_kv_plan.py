"""The cut of the launches over the paged cache, checked on the host over the admitted sizes."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "w8a8_quantized_linear_channel_amd", "csrc")


def test_every_launch_is_within_its_limits(tmp_path):
    exe = str(tmp_path / "kv_plan_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}",
                    os.path.join(HERE, "native", "kv_plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
