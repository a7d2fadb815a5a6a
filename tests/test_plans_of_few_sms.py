"""CPU-only: plans for one and for a few SMs, where there is no room for pairs of blocks."""
import os
import subprocess
import sys

import pytest

import dense_fp32_matrix_08_gb300 as sg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = (1, 3, 40, 300, 5000)


def test_one_sm_does_not_end_the_process():
    """In a process of its own, which a division by zero would end."""
    code = "import dense_fp32_matrix_08_gb300 as sg; print(sg.i8_linear_plan(40, 300, 2000, num_sms=1))"
    assert subprocess.run([sys.executable, "-c", code], capture_output=True, cwd=ROOT).returncode == 0


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 152])
def test_integer_product(sms):
    for M in SIZES:
        for N in (1, 300, 4096):
            for K in (1, 700, 131071):
                plan = sg.i8_linear_plan(M, N, K, sms)
                assert (plan["tile_tokens"] == 0) == (M <= 2)
                if sms == 1:
                    assert plan["tile_channels"] in (0, 128)
                assert plan["split"] <= max(1, sms)


def test_one_sm_does_not_end_the_process_of_the_8_bit_float_product():
    code = "import dense_fp32_matrix_08_gb300 as sg; print(sg.f8_gemm_plan(40, 300, 2000, num_sms=1))"
    assert subprocess.run([sys.executable, "-c", code], capture_output=True, cwd=ROOT).returncode == 0


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 152])
def test_8_bit_float_product(sms):
    for M in SIZES:
        for N in (1, 300, 4096):
            for K in (1, 700, 131071):
                plan = sg.f8_gemm_plan(M, N, K, num_sms=sms)
                if sms == 1:
                    assert plan["tile_cols"] < 256
                assert plan["split"] <= max(1, sms)
