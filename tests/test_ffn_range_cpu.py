"""The feed-forward half's calls at the ends of what they take: workspaces and refusals, without a GPU."""

import pytest

import kernelized_causal_self_gb300 as la
from kernelized_causal_self_gb300 import build as labuild


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def test_parts_of_cut_sums_are_bounded(lib):
    """Workspaces of bf16 gradients have room for parts of 32768 terms at most: of tokens, and of dx's 2 F."""
    for T, C, F in ((1 << 20, 1024, 2560), (1 << 24, 8, 8), (40000, 2560, 5120), (4096, 4096, 65536)):
        dact = -(-4 * T * F // 256) * 256
        floats = (la.la_ffn_gate_backward_workspace_bytes(T, C, F) - 256 - dact) // 4
        parts_w, parts_x = -(-T // 32768), -(-2 * F // 32768)
        need = (2 * parts_w * F * C if parts_w > 1 else 0) + (parts_x * T * C if parts_x > 1 else 0)
        assert floats >= need
