"""Arguments of the stalled producer of the paged chunk kernel (no GPU needed)."""
import pytest

llb = pytest.importorskip("decoder_only_transformer_llama_b200",
                          reason="library not built (run decoder_only_transformer_llama_b200/build.py)")
L = llb.lib()


def test_arguments_are_checked():
    for which, unit, ns in ((1, 0, 10000), (2, 0, 10000), (4, 0, 10000), (-1, 0, 10000), (3, -1, 10000), (3, 0, 999),
                            (3, 0, 2_000_000_001)):
        assert L.llama_debug_stall(None, which, unit, ns) == llb.LLAMA_ERR_INVALID_ARG and llb.last_error()
    with pytest.raises(llb.LlamaError):
        llb.paged_debug_stall(-2)
    with pytest.raises(llb.LlamaError):
        llb.paged_debug_stall(0, wait_limit_ns=10)


def test_armed_and_disarmed():
    llb.paged_debug_stall(3, wait_limit_ns=2_000_000_000)
    llb.paged_debug_stall(-1)
