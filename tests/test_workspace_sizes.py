"""The binding asks the library for a shape's workspace once, and keeps a bounded number of answers: a server's M takes
every value."""
import pytest

import fp8_group_quant_amd as fq
from test_serving_abi import no_gpu


class Library:
    """Sizes by shape, and how often one was asked for."""

    def __init__(self):
        self.asked = 0

    def fp8q_gemm_workspace_size(self, *shape):
        self.asked += 1
        return sum(shape)

    fp8q_gemm_mxfp4_workspace_size = fp8q_gemm_workspace_size


@no_gpu
@pytest.mark.parametrize("name,more", [("_gemm_workspace_size", (0,)), ("_gemm_mxfp4_workspace_size", ())])
def test_sizes_that_are_kept_are_bounded(monkeypatch, name, more):
    lib, size = Library(), getattr(fq, name)
    monkeypatch.setattr(fq, "load_library", lambda: lib)
    size.cache_clear()
    try:
        most = size.cache_info().maxsize
        for m in range(1, most + 1000):
            assert size(0, m, 128, 256, *more) == m + 128 + 256
        assert size.cache_info().currsize == most
        lib.asked = 0
        assert size(0, most, 128, 256, *more) == most + 128 + 256 and lib.asked == 0
        assert size(0, 1, 128, 256, *more) == 1 + 128 + 256 and lib.asked == 1
        assert size(1, most, 128, 256, *more) == most + 128 + 256 and lib.asked == 2  # another GPU's
    finally:
        size.cache_clear()


@no_gpu
def test_nothing_else_of_the_binding_grows():
    """No container of the module but the fixed tables."""
    held = {k for k, v in vars(fq).items() if isinstance(v, (dict, list, set)) and not k.startswith("__")}
    assert held == {"_SIGNATURES", "_DTYPES", "_SCALE_FMT"}
