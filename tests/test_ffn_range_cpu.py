"""The feed-forward half's calls at the ends of what they take: workspaces and refusals, without a GPU."""

import pytest
import torch

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


def test_sizes_past_32_bits_are_refused(lib):
    """They were cut to their low 32 bits: 2^32 + 5 rows arrived in the library as 5."""
    many = (1 << 32) + 5

    def t(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")
    w, wide = t(8, 8), t(8, many + 3)
    x, h, long = t(many, 8), t(many, 8), t(2, many + 3)
    kept = t(many, 2, 8, dtype=torch.int8), t(many, 2, 1, dtype=torch.uint8)
    codes = t(2, many + 3, dtype=torch.int8), t(2, -(-many // 32), dtype=torch.uint8)
    before = la.la_kernel_launches()
    for call in (lambda: la.la_ffn_gate(x, w, w), lambda: la.la_ffn_gate(x, w, w, checkpoint=kept),
                 lambda: la.la_ffn_gate(x, w, w, out=h),
                 lambda: la.la_ffn_gate_backward(x, w, w, h), lambda: la.la_ffn_gate_backward(x, w, w, h, dx=x),
                 lambda: la.la_ffn_gate(long, wide, wide), lambda: la.la_ffn_gate(t(2, 8), x, x),
                 lambda: la.la_ffn_gate_backward(t(2, 8), x, x, t(2, many)),
                 lambda: la.la_checkpoint(long), lambda: la.la_layer_norm(long, long[0]),
                 lambda: la.la_layer_norm_backward(long, long[0], long),
                 lambda: la.la_layer_norm_backward(codes, long[0], long),
                 lambda: la.la_checkpoint_restore(*codes, out=long),
                 lambda: la.la_layer_norm_workspace_bytes(4, many + 3),
                 lambda: la.la_ffn_gate_workspace_bytes(many, 8, 8),
                 lambda: la.la_ffn_gate_workspace_bytes(4, 8, many + 3),
                 lambda: la.la_ffn_gate_backward_workspace_bytes(4, many + 3, 8),
                 lambda: la.la_ffn_gate_backward_workspace_bytes(-many, 8, 8)):
        with pytest.raises(ValueError, match="past 32 bits"):
            call()
    assert la.la_kernel_launches() == before
