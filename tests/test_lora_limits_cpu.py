"""CPU: sizes at the ends of what the adapter calls accept. Nothing here reaches
a GPU."""
from test_lora_cpu import L, backward  # noqa: F401


def test_gradient_limit_counts_the_padded_outputs(L):
    """dY's rows in the workspace have N rounded up to 128 columns: those are
    what the 32-bit offsets (512·N below 2^31) have to hold."""
    for T in (40, 321):
        for N in ((1 << 22) - 8, (1 << 22) - 120):
            assert backward(L, T=T, N=N, K=128) == L.AWQ_E_UNSUPPORTED
            assert "32-bit offsets" in L.last_error()
        assert backward(L, T=T, N=(1 << 22) - 128, K=128, wsb=16) == L.AWQ_E_WORKSPACE
