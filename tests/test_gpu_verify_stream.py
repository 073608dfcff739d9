"""Log probabilities of a verify handle whose stream is not the current one."""
import pytest
import torch

import spec_inputs as si
import speculative_decoding_verification_22_gb300 as sv

pytestmark = pytest.mark.gpu


def engine(stream, K=3, V=3000):
    """A handle on `stream` that has run a round, its tokens, and what its log
    probabilities are when the stream is the current one."""
    wl = si.workload("tiny", dtype="bf16", B=2, K=K, V=V, d=256)
    W = si.make_weights(wl, seed=3, device="cuda")
    inp = si.make_round(wl, W, seed=4, T=1.0)
    torch.cuda.synchronize()
    eng = sv.SpecVerify(wl.V, wl.d, wl.B, wl.K, wl.dtype, stream=stream)
    with torch.cuda.stream(stream):
        tokens, _ = eng.run(inp["hidden"], W, inp["draft"], inp["q_logits"], inp["uniforms"], 1.0)
        want = eng.log_probs(tokens, 7)
    torch.cuda.synchronize()
    return eng, tokens, want


def same(a, b):
    return all(torch.equal(x.view(torch.int32), y.view(torch.int32)) for x, y in zip(a, b))


def test_outputs_are_not_memory_that_the_current_stream_still_uses():
    """A block that was freed on the current stream, whose kernels write it later."""
    eng, tokens, want = engine(torch.cuda.Stream())
    for _ in range(3):
        old = [torch.empty_like(o) for o in want]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for o in old:
            o.fill_(7)
        places = {o.data_ptr() for o in old}
        del old, o
        got = eng.log_probs(tokens, 7)
        assert not places & {o.data_ptr() for o in got}
        torch.cuda.synchronize()
        assert same(got, want)
        del got
    assert eng.status() == sv.SV_OK
    eng.close()


def test_dropped_outputs_are_not_handed_to_the_current_stream():
    stream = torch.cuda.Stream()
    eng, tokens, want = engine(stream)
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
    got = eng.log_probs(tokens, 7)  # behind the sleep
    places = {o.data_ptr() for o in got}
    del got
    new = [torch.full_like(o, 3) for o in want]
    assert not places & {o.data_ptr() for o in new}
    torch.cuda.synchronize()
    assert all((o == 3).all() for o in new)
    eng.close()


def test_given_outputs_and_another_stream_set_later():
    eng, tokens, want = engine(torch.cuda.Stream())
    for stream in (torch.cuda.Stream(), torch.cuda.default_stream()):
        sv.spec_verify_set_stream(eng.h, stream)
        assert sv.spec_verify_stream(eng.h) == stream.cuda_stream
        outs = [torch.zeros_like(o) for o in want]
        torch.cuda.synchronize()
        got = eng.log_probs(tokens, 7, out=outs)
        assert all(a is b for a, b in zip(got, outs))
        torch.cuda.synchronize()
        assert same(got, want) and same(eng.log_probs(tokens, 7), want)
        outs = [None] + outs[1:]
        assert eng.log_probs(top=7, out=outs)[0] is None
        torch.cuda.synchronize()
        assert same(outs[1:], want[1:])
    for bad in (outs[:2], [tokens] + outs[1:], outs[1:] + outs[:1],
                [want[0].t().contiguous().t()] + outs[1:]):
        with pytest.raises(ValueError):
            eng.log_probs(tokens, 7, out=bad)
    eng.close()


def test_outputs_of_a_run_and_of_a_tree_belong_to_the_handle_too():
    wl = si.workload("tiny", dtype="bf16", B=2, K=3, V=3000, d=256)
    W = si.make_weights(wl, seed=3, device="cuda")
    inp = si.make_round(wl, W, seed=4, T=1.0)
    torch.cuda.synchronize()
    eng = sv.SpecVerify(wl.V, wl.d, wl.B, wl.K, wl.dtype, stream=torch.cuda.Stream())
    args = inp["hidden"], W, inp["draft"], inp["q_logits"], inp["uniforms"], 1.0
    tokens = inp["draft"].view(wl.B, wl.K)
    parents = torch.arange(-1, wl.K - 1, dtype=torch.int32, device="cuda").repeat(wl.B, 1)
    calls = (lambda: eng.run(*args), lambda: eng.run_truncated(*args, target_top_k=50),
             lambda: eng.run_tree_greedy(inp["hidden"], W, tokens, parents))
    for call in calls:
        got = call()
        torch.cuda.synchronize()
        want = [t.clone() for t in got]
        old = [torch.empty_like(t) for t in got]
        places = {o.data_ptr() for o in old}
        torch.cuda._sleep(20_000_000)
        for o in old:
            o.fill_(7)
        del old, o, got
        got = call()
        assert not places & {t.data_ptr() for t in got}
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    mine = torch.empty(wl.B, dtype=torch.int32, device="cuda")
    assert eng.run(*args, out_n_accepted=mine)[1] is mine
    torch.cuda.synchronize()
    assert eng.status() == sv.SV_OK
    eng.close()
