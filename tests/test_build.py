"""The build's check of kernels whose register split fixes their register count."""
import pytest

from gemm_iq2_ks_b200 import build

REPORT = """ptxas info    : Compiling entry function '_ZN3iqk6k_topkEv' for 'sm_100a'
ptxas info    : Function properties for _ZN3iqk6k_topkEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 40 registers, used 0 barriers
ptxas info    : Compiling entry function '_ZN3iqk10k_fp8_gemmILi128ELb0ELb0EEEv' for 'sm_100a'
ptxas info    : Function properties for _ZN3iqk10k_fp8_gemmILi128ELb0ELb0EEEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 1 barriers
"""


def test_register_counts_are_checked():
    build.check_registers(REPORT.format(96))
    with pytest.raises(RuntimeError, match="88 registers"):
        build.check_registers(REPORT.format(88))
