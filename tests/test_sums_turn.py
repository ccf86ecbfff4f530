"""The fp8 experts' issuer waits for all readers of a buffer of sums before the next block's products go there: every
sequence of tiles is checked on the host, with the code that the kernel uses."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_get_dispatch_layout_gb300", "csrc")


def test_no_sums_are_overwritten_before_they_are_read(tmp_path):
    exe = str(tmp_path / "sums_turn_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                    os.path.join(HERE, "sums_turn_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
