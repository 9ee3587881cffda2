"""The diagnostic of the norm's waits is taken by the next call that launches, and not by one that is refused or empty (no GPU needed)."""
import nvfp4_quantization_current_gb300 as Q
from test_abi import status_of
from test_norm_abi import add_args, grad_args
from test_operators_abi import L  # noqa: F401 (a fixture)


def test_taken_once_and_cleared(L):
    try:
        assert L.selftest_norm_give_up(1) == Q.Q_OK
        assert status_of(L, "norm_add", *add_args(M=0, x=None, r=None, w=None, h=None, y=None, s=None))[0] == Q.Q_OK
        assert status_of(L, "norm_grad", *grad_args(K=0))[0] == Q.Q_ERR_SHAPE
        assert L.q_selftest_inject_launch_error(1) == Q.Q_OK
        assert status_of(L, "norm_grad", *grad_args())[0] == Q.Q_ERR_CUDA
    finally:
        L.q_selftest_inject_launch_error(0)
        assert L.selftest_norm_give_up(0) == Q.Q_OK
