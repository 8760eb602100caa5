"""CPU check, on stand-ins for CUDA tensors and streams (fake_cuda), that the verification calls make their workspaces and
outputs on the stream that they run on."""
import pytest
import torch

import fake_cuda as fc
import speculative_decoding_verification_target_gb300 as sv

B, K, V, N = 2, 3, 64, 2


def t(*shape, dtype=torch.float32):
    return fc.Tensor(shape, dtype)


def arguments():
    return t(B, K + 1, V), t(B, K, V), t(B, K, dtype=torch.int32), t(B, dtype=torch.int64)


CALLS = {
    "verify": lambda **kw: sv.verify(*arguments(), **kw),
    "cactus_verify": lambda **kw: sv.cactus_verify(*arguments(), 0.1, **kw),
    "greedy_verify": lambda **kw: sv.greedy_verify(t(B, K + 1, V), t(B, K, dtype=torch.int32), **kw),
    "verify_filtered": lambda **kw: sv.verify_filtered(*arguments(), top_k=4, **kw),
    "counterfactual_gamma": lambda **kw: sv.counterfactual_gamma(t(B, K + 1, V), t(N, B, K, V), 1.0, 0, *arguments()[2:], **kw),
    "accept_length_estimate": lambda **kw: sv.accept_length_estimate(t(N, B, K), **kw),
    "HedgeFeedback": lambda **kw: sv.HedgeFeedback(N, B, K, **kw),
}


@pytest.fixture
def fake(monkeypatch):
    return fc.install(monkeypatch, sv)


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_is_made_on_its_stream(fake, name):
    torch_, lib = fake
    here, s = torch_.cuda.now, fc.Stream("given")
    CALLS[name](stream=s)
    assert torch_.made and all(x.made_on is s and x.used_on == [here] for x in torch_.made)
    assert lib.calls[-1][1][-1].value == s.cuda_stream and torch_.cuda.now is here


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_serves(fake, name):
    torch_, lib = fake
    CALLS[name]()
    assert torch_.made and all(x.made_on is torch_.cuda.now and x.used_on == [] for x in torch_.made)
    assert lib.calls[-1][1][-1].value == torch_.cuda.now.cuda_stream


def test_feedback_weights_can_be_read_on_the_current_stream_at_once(fake):
    torch_, _ = fake
    s = fc.Stream("given")
    sv.HedgeFeedback(N, B, K, stream=s)
    assert torch_.cuda.now.waited_for == [s]
