"""Log probabilities of a round's tokens from the verify step's own logits."""
import pytest
import torch

import spec_inputs as si
import speculative_decoding_verification_22_gb300 as sv
from layer_common import log_probs_error, log_probs_ref
from target_common import within

pytestmark = pytest.mark.gpu


def check(eng, got, tokens, top, T):
    logits = eng.logits()
    R, V = logits.shape
    t = (tokens if tokens is not None else torch.full((R, 1), -1, device="cuda")).reshape(R, 1)
    want = log_probs_ref(logits, t, top, T)
    if tokens is not None:
        within(got[0].view(R, 1), want[0], log_probs_error(want[0], V))
    else:
        assert got[0] is None
    within(got[1].view(R), want[1], want[1].abs() * (V / 256 + 64) * 2.0 ** -22
           + (V / 256 + 64) * 2.0 ** -24)
    if top:
        assert torch.equal(got[2].view(R, top), want[2])
        within(got[3].view(R, top), want[3], log_probs_error(want[3], V))


@pytest.mark.parametrize("over,T", [(dict(dtype="fp32", B=2, K=4), 1.0),
                                    (dict(dtype="bf16", B=3, K=3, V=1000), 0.7),
                                    (dict(dtype="bf16", B=8, K=7, V=5003), 0.0),
                                    (dict(dtype="bf16", B=1, K=0, V=40000), 1.0)])
def test_tokens_of_a_round(over, T):
    """What was emitted, and -1 behind it: each token's log probability is that of
    its own row, and equals the alternatives' where it is one of them."""
    wl = si.workload("tiny", **(dict(V=1000, d=256) | over))
    W = si.make_weights(wl, seed=7, device="cuda")
    inp = si.make_round(wl, W, seed=8, T=T)
    eng = sv.SpecVerify(wl.V, wl.d, wl.B, wl.K, wl.dtype)
    with pytest.raises(sv.SpecVerifyError):
        eng.log_probs(top=1)  # nothing has run
    tokens, n = eng.run(inp["hidden"], W, inp["draft"], inp["q_logits"], inp["uniforms"], T)
    for top, at in ((0, 1.0), (5, 1.0), (20, 0.8)):
        got = eng.log_probs(tokens, top, at)
        check(eng, got, tokens, top, at)
        after = torch.arange(wl.K + 1, device="cuda")[None] > n[:, None]
        assert (got[0][after] == 0).all() and (got[0][~after] < 0).all()
        if top:
            same = got[2] == tokens[..., None]
            assert torch.equal(got[3][same], got[0][same.any(-1)])
        if T == 0 and top:  # a greedy round: the emitted token is the first alternative
            assert torch.equal(got[2][..., 0][~after], tokens[~after])
    check(eng, eng.log_probs(top=3), None, 3, 1.0)
    assert eng.status() == sv.SV_OK
    again, _ = eng.run(inp["hidden"], W, inp["draft"], inp["q_logits"], inp["uniforms"], T)
    assert torch.equal(again, tokens)  # the scoring left the handle as it was
    eng.close()


def test_a_token_outside_the_vocabulary_is_reported():
    wl = si.workload("tiny", dtype="bf16", B=2, K=2, V=1000, d=256)
    W = si.make_weights(wl, seed=1, device="cuda")
    inp = si.make_round(wl, W, seed=2, T=1.0)
    eng = sv.SpecVerify(wl.V, wl.d, wl.B, wl.K, wl.dtype)
    tokens, _ = eng.run(inp["hidden"], W, inp["draft"], inp["q_logits"], inp["uniforms"], 1.0)
    bad = torch.full_like(tokens, 5)
    bad[1, 1] = wl.V
    got = eng.log_probs(bad)[0]
    assert torch.isnan(got[1, 1]) and torch.isfinite(got).sum() == bad.numel() - 1
    assert eng.status() == sv.SV_ERR_TOKEN and eng.status() == sv.SV_OK
    eng.close()


def test_log_probs_of_an_fp8_head_and_of_a_captured_round():
    """Rounds and their scoring captured together and replayed on other inputs."""
    wl = si.workload("tiny", dtype="bf16", B=2, K=3, V=3000, d=256)
    W = si.make_weights(wl, seed=3, device="cuda")
    first, second = (si.make_round(wl, W, seed=s, T=1.0) for s in (4, 5))
    stream = torch.cuda.Stream()
    eng = sv.SpecVerify(wl.V, wl.d, wl.B, wl.K, wl.dtype, stream=stream)
    tokens = torch.empty(wl.B, wl.K + 1, dtype=torch.int32, device="cuda")
    n = torch.empty(wl.B, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def step():
        eng.run(first["hidden"], W, first["draft"], first["q_logits"], first["uniforms"], 1.0,
                tokens, n)
        return eng.log_probs(tokens, 4)
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    for k in first:
        if torch.is_tensor(first[k]):
            first[k].copy_(second[k])
    graph.replay()
    torch.cuda.synchronize()
    check(eng, got, tokens, 4, 1.0)
    assert eng.status() == sv.SV_OK
    eng.close()
    W8, ws = si.quantize_rows_e4m3(W)
    h8, hs = si.quantize_rows_e4m3(first["hidden"].reshape(-1, wl.d))
    eng = sv.SpecVerify(wl.V, wl.d, wl.B, wl.K, "fp8")
    tokens, _ = eng.run_fp8(h8.view(wl.B, wl.K + 1, wl.d), hs.view(wl.B, wl.K + 1), W8, ws,
                            first["draft"], None, first["uniforms"], 1.0)
    check(eng, eng.log_probs(tokens, 7, 0.9), tokens, 7, 0.9)
    eng.close()
