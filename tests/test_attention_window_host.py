"""Windows of any size in the binding's plans, without a device."""
import pytest

import implicit_gemm_dgrad_gb300 as cdg


def test_windows_past_32_bits_are_windows():
    for window in ((1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 1, 1 << 70):
        far, plain = (cdg.attention_plan_host(4, 2, 64, window=w) for w in (window, 0))
        for sizes in ((1, 8192, 1), (3000, 3000, 2)):
            assert far.workspace_bytes(*sizes) == plain.workspace_bytes(*sizes)
            assert far.grad_workspace_bytes(*sizes) == plain.grad_workspace_bytes(*sizes)
        with pytest.raises(cdg.CdgError):  # with no causal mask a window is refused, whatever its lower bits say
            cdg.attention_plan_host(4, 2, 64, causal=False, window=window)
    for window in (-1, -(1 << 31), -(1 << 32)):
        with pytest.raises(cdg.CdgError):
            cdg.attention_plan_host(4, 2, 64, window=window)
