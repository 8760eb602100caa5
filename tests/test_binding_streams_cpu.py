"""CPU check, on stand-ins for CUDA tensors and streams (fake_cuda), that the verification calls make their workspaces and
outputs on the stream that they run on."""
import sys

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


# what each call looks at: its inputs, in the order that CALLS makes them, and what may be given to it
INPUTS = {"verify": range(4), "cactus_verify": range(4), "greedy_verify": range(2), "verify_filtered": range(4),
          "counterfactual_gamma": (0, 1, 4, 5), "accept_length_estimate": range(1)}
GIVEN = {"accept_len": (B,), "out_tokens": (B, K + 1), "diag": (B, K, 4), "workspace": (1 << 15,), "gamma_star": (B, K),
         "gamma": (N, B, K), "loss": (N, B, K), "est": (N, B)}
TAKES = {"verify": "accept_len out_tokens diag workspace", "cactus_verify": "accept_len out_tokens diag gamma_star workspace",
         "greedy_verify": "accept_len out_tokens workspace", "verify_filtered": "accept_len out_tokens diag workspace",
         "counterfactual_gamma": "gamma loss accept_len out_tokens diag workspace", "accept_length_estimate": "est loss"}


@pytest.mark.parametrize("where,words", [(1, "must be on cuda:0, got cuda:1"), (-1, "must be a CUDA tensor")])
@pytest.mark.parametrize("name,i", [(n, i) for n, which in INPUTS.items() for i in which])
def test_inputs_elsewhere_are_refused(fake, monkeypatch, name, i, where, words):
    _, lib = fake
    made = iter(range(100))
    monkeypatch.setattr(sys.modules[__name__], "t", lambda *shape, dtype=torch.float32: fc.Tensor(shape, dtype, where if next(made) == i else 0))
    with pytest.raises(ValueError, match=words):
        CALLS[name]()
    assert lib.calls == []


@pytest.mark.parametrize("where,words", [(1, "must be on cuda:0, got cuda:1"), (-1, "must be a CUDA tensor")])
@pytest.mark.parametrize("name,given", [(n, g) for n, gs in TAKES.items() for g in gs.split()])
def test_outputs_and_workspaces_elsewhere_are_refused(fake, name, given, where, words):
    _, lib = fake
    dtype = torch.uint8 if given == "workspace" else torch.int32 if given in ("accept_len", "out_tokens") else torch.float32
    there = fc.Tensor(GIVEN[given], dtype)
    CALLS[name](**{given: there})
    assert there.address in [getattr(x, "value", None) for x in lib.calls[-1][1]]
    del lib.calls[:]
    with pytest.raises(ValueError, match=words):
        CALLS[name](**{given: fc.Tensor(GIVEN[given], dtype, where)})
    assert lib.calls == []
