"""The stream of a verify handle and the outputs of its log probabilities, without a GPU."""
import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_22_gb300 import build as b
    b.build()
    return sv.load_library()


def test_a_null_handle_has_no_stream(lib):
    assert sv.spec_verify_stream(None) == 0


def test_outputs_that_do_not_fit_are_refused():
    eng = sv.SpecVerify.__new__(sv.SpecVerify)  # no GPU, no handle
    eng.B, eng.K, eng.V, eng.h, eng.device = 2, 3, 40, None, torch.device("cuda", 0)
    f32 = torch.zeros(2, 4)  # not on the GPU
    for out, top in (([], 0), ([None], 0), ([f32, f32], 0), ([None, None], 0), ([None, f32], 0),
                     ([None, f32], 2), ([None, None, None, None], 2)):
        with pytest.raises(ValueError):
            eng.log_probs(top=top, out=out)
