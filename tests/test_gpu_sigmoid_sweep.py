"""The experts' sigmoid and silu on every one of the 2^32 fp32 numbers against 64 bits."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_get_dispatch_layout_gb300", "csrc")


@pytest.mark.gpu
def test_sigmoid_and_silu_of_all_fp32_numbers(tmp_path):
    so = str(tmp_path / "libsigmoid_sweep.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-shared",
                    "-Xcompiler", "-fPIC", "-I", CSRC, "-o", so, os.path.join(HERE, "sigmoid_sweep.cu")], check=True, capture_output=True)
    lib = ctypes.CDLL(so)
    lib.sigmoid_sweep.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    worst = torch.zeros(3, dtype=torch.int64, device="cuda")
    assert lib.sigmoid_sweep(worst.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    sigmoid, silu, wrong = worst.cpu().numpy().view(np.float64)[:2].tolist() + [int(worst[2])]
    print(f"sigmoid within {sigmoid * 2 ** 23:.2f} * 2^-23 of itself, silu within {silu * 2 ** 23:.2f}")
    assert wrong == 0
    # 2^t: 2^-22; the rest of t, its product and that with 2^t: a rounding each; 1 + exp: one; the reciprocal: 2^-23; silu: its product
    assert sigmoid <= 2.0 ** -22 + 4 * 2.0 ** -24 + 2.0 ** -23
    assert silu <= sigmoid + 2.0 ** -24 * (1 + 2.0 ** -20)
