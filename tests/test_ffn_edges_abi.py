"""CPU checks of the feed-forward entry points at their edges: calls that are
accepted or refused before any HIP call."""
from test_ffn_abi import INVALID, L, P, gated_bwd, linear_bwd  # noqa: F401


def test_backward_without_rows_or_weight_gradients(L):
    """M == 0 and the input's gradient alone is a no-op, also with the null
    address of an empty tensor; with rows, nothing to compute is refused."""
    for dA in (P, None):
        assert linear_bwd(L, M=0, A=None, d=None, dA=dA, dB=None, ws=None, wsb=0) == 0
        assert gated_bwd(L, M=0, A=None, d=None, dA=dA, dG=None, dU=None, ws=None, wsb=0) == 0
    assert linear_bwd(L, M=1, dA=None, dB=None) == INVALID
    assert gated_bwd(L, M=1, dA=None, dG=None, dU=None) == INVALID
    assert linear_bwd(L, M=0, dA=None, dB=None, N=60) == INVALID
    assert gated_bwd(L, M=0, dA=None, dG=P, dU=None) == INVALID
