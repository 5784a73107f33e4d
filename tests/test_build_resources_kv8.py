"""Register-spill budgets of the 8-bit operators' kernels, from ptxas's report of
the library's own compile (no GPU)."""
import pytest

from tests.test_build_resources import report  # noqa: F401  (the module's fixture)

BUDGETS = [
    ("_ZN6mixllm11w8a8_kernel", 0),
    ("_ZN6mixllm16w8a8_pair_kernel", 0),
    ("_ZN6mixllm19row_quantize_kernelI6__half", 0),
    ("_ZN6mixllm19row_quantize_kernelIf", 64),  # offline
    ("_ZN6mixllm17kv8_decode_kernel", 0),
    ("_ZN6mixllm17kv8_append_kernel", 128),  # three blocks an SM with them, two without: 42 against 46 us for a prompt
    ("_ZN6mixllm15kv8_read_kernel", 0),
    ("_ZN6mixllm21head_norm_rope_kernel", 0),
]


@pytest.mark.parametrize("prefix,budget", BUDGETS, ids=[p for p, _ in BUDGETS])
def test_spill_loads_within_budget(report, prefix, budget):  # noqa: F811
    found = {k: v for k, v in report.items() if k.startswith(prefix)}
    assert found, prefix
    for name, loads in found.items():
        assert loads <= budget, f"{name}: {loads} bytes of spill loads, budget {budget}"
