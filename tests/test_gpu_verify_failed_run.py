"""Log probabilities after a run that could not be enqueued."""
import ctypes

import pytest
import torch

import spec_inputs as si
import speculative_decoding_verification_22_gb300 as sv

pytestmark = pytest.mark.gpu

RELAXED = 2  # capture mode


class Capture:
    """A capture on a blocking stream, during which a launch on the legacy default stream
    is refused on the host (an implicit dependency); what was captured is dropped."""

    def __init__(self):
        self.cuda = ctypes.CDLL("libcuda.so.1")
        self.stream = ctypes.c_void_p()
        assert self.cuda.cuStreamCreate(ctypes.byref(self.stream), 0) == 0

    def __enter__(self):
        assert self.cuda.cuStreamBeginCapture_v2(self.stream, RELAXED) == 0

    def __exit__(self, *what):
        graph = ctypes.c_void_p()
        self.cuda.cuStreamEndCapture(self.stream, ctypes.byref(graph))
        if graph:
            self.cuda.cuGraphDestroy(graph)
        self.cuda.cuStreamDestroy_v2(self.stream)


def refused(call, code):
    with pytest.raises(sv.SpecVerifyError) as e:
        call()
    assert e.value.code == code


def test_a_run_that_failed_has_no_log_probabilities():
    wl = si.workload("tiny", dtype="bf16", B=2, K=3, V=1000, d=256)
    W = si.make_weights(wl, seed=1, device="cuda")
    inp = si.make_round(wl, W, seed=2, T=1.0)
    eng = sv.SpecVerify(wl.V, wl.d, wl.B, wl.K, wl.dtype, stream=torch.cuda.default_stream())
    tokens = torch.empty(wl.B, wl.K + 1, dtype=torch.int32, device="cuda")
    n = torch.empty(wl.B, dtype=torch.int32, device="cuda")
    outs = [torch.empty(wl.B, wl.K + 1, device="cuda") for _ in range(2)]

    def run(T=1.0):
        eng.run(inp["hidden"], W, inp["draft"], inp["q_logits"], inp["uniforms"], T, tokens, n)

    def score():
        return eng.log_probs(tokens, out=outs)
    torch.cuda.synchronize()
    for first in (True, False):
        with Capture():
            refused(run, sv.SV_ERR_CUDA)
        refused(score, sv.SV_ERR_ARG)
        run()
        want = score()[0].clone()
        torch.cuda.synchronize()
        assert (want <= 0).all() and (want < 0).any()
    # what is refused before anything is enqueued leaves the last run as it was
    refused(lambda: run(float("nan")), sv.SV_ERR_ARG)
    assert torch.equal(score()[0], want)
    assert eng.status() == sv.SV_OK
    eng.close()
