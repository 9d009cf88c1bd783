"""CPU: the test hook of the attention's bounded waits checks its arguments."""
from fp4_weight_only_nvfp4_gb300 import _lib


def test_arguments():
    from fp4_weight_only_nvfp4_gb300 import build
    build.build()
    f = _lib.lib().vt_fp4_attention_test_hooks
    assert f(-1, 0) == _lib.VT_ERR_INVALID_ARG and f(0, -2 ** 31) == _lib.VT_ERR_INVALID_ARG
    assert f(20000, 3) == _lib.VT_OK and f(20000, -3) == _lib.VT_OK
    assert f(0, 0) == _lib.VT_OK
