"""CPU checks of what the drafting operators refuse beyond shapes and pointers."""
import gemm_epilogue_transformer_bf16_gb300 as coda


def test_the_status_of_rows_that_are_no_probabilities_has_a_name():
    from gemm_epilogue_transformer_bf16_gb300 import _build
    _build.build()
    assert coda.status_string(12) == "CODA_ERR_PROBABILITY_RANGE"
