"""Register-spill budgets of the KV-cache and norm kernels, from ptxas's report
of the library's own compile (no GPU)."""
import pytest

from tests.test_build_resources import report  # noqa: F401  (the module's fixture)

BUDGETS = [
    ("_ZN6mixllm17kv4_decode_kernelILi128ELi1E", 64),
    ("_ZN6mixllm17kv4_decode_kernelILi128ELi2E", 64),
    ("_ZN6mixllm17kv4_decode_kernelILi64ELi1E", 0),
    ("_ZN6mixllm17kv4_decode_kernelILi64ELi2E", 320),
    ("_ZN6mixllm17kv4_prompt_kernel", 256),  # outside the softmax's loop
    ("_ZN6mixllm22kv4_prompt_join_kernel", 0),
    ("_ZN6mixllm22kv4_prompt_plan_kernel", 0),
    ("_ZN6mixllm17kv4_append_kernel", 256),
    ("_ZN6mixllm15kv4_read_kernel", 0),
    ("_ZN6mixllm17kv4_assign_kernel", 0),
    ("_ZN6mixllm20residual_norm_kernel", 0),
    ("_ZN6mixllm21dequantize_act_kernel", 0),
]


@pytest.mark.parametrize("prefix,budget", BUDGETS, ids=[p for p, _ in BUDGETS])
def test_spill_loads_within_budget(report, prefix, budget):  # noqa: F811
    found = {k: v for k, v in report.items() if k.startswith(prefix)}
    assert found, prefix
    for name, loads in found.items():
        assert loads <= budget, f"{name}: {loads} bytes of spill loads, budget {budget}"
