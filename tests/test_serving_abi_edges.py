"""More refusals of the serving entry points, before any CUDA call (no GPU)."""
import pytest

import quantized_expert_ffn_bias_gb300 as coli
from tests.test_serving_abi import attn, built, kv, refused  # noqa: F401  (a fixture)


def test_kv_debug_inject_arguments():
    refused(coli.COLI_EINVAL, coli.colibri_kv_debug_inject, coli.COLI_INJECT_BAD_EXPERT_ID, 1.0)
    refused(coli.COLI_EINVAL, coli.colibri_kv_debug_inject, -1, 1.0)
    refused(coli.COLI_EINVAL, coli.colibri_kv_debug_inject, 0, float("nan"))
    for ms in (2.0, -1.0, 1e-9, float("inf"), 0.0):
        coli.colibri_kv_debug_inject(0, ms)


@pytest.mark.parametrize("scale", [2.4e38, -3.0e38, 3.4e38, float("-inf"), float("nan")])
def test_attention_scale_out_of_range(scale):
    """The kernel multiplies with scale log2(e), which has to be finite."""
    refused(coli.COLI_EINVAL, lambda: attn(kv(), scale=scale))
