"""The switch of the linear layer's self-test: declared, exported and off at first."""
from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build


def test_declared_and_exported():
    build.build()
    assert "moe_selftest_give_up" in B.declared_functions() and hasattr(B.lib(), "moe_selftest_give_up")
    B.moe_selftest_give_up(True)
    B.moe_selftest_give_up(False)
