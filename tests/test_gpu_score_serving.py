"""The serving example with the operators between its last layer and the verification: 8-bit products, penalties and a mask."""
import os
import sys

import pytest
import torch

import score_util as su
import speculative_decoding_verification_target_gb300 as sv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def bits(allowed):
    """Allowed tokens as a mask of 32-bit words."""
    words = (allowed.view(-1, 32).long() << torch.arange(32)).sum(1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().cuda()


@pytest.mark.parametrize("kw", [dict(int8=True), dict(penalties=dict(repetition=1.3, frequency=0.2, presence=0.1)),
                                dict(int8=True, penalties=dict(frequency=0.4), window=70)])
def test_serving(kw):
    import serve_drafts as ex
    prompt = [100, 64, 5, 130]
    cache, target, text, accepted = ex.serve(rounds=10, prompts=prompt, **kw)
    assert cache.status() == 0 and all(sv.read_status(w) == 0 for w in target._product_ws.values())
    assert bool(target._product_ws) == kw.get("int8", False)
    assert cache.lengths.tolist() == [len(t) - 1 for t in text]
    for s, n in enumerate(prompt):
        assert len(text[s]) == n + sum(a[s] + 1 for a in accepted)


def test_a_masked_token_never_comes():
    import serve_drafts as ex
    allowed = torch.rand(2048, generator=torch.Generator().manual_seed(3)) < 0.3
    prompt = [20, 7, 33, 64]
    _, _, text, _ = ex.serve(rounds=12, prompts=prompt, allowed=bits(allowed), penalties=dict(repetition=1.1))
    for t, n in zip(text, prompt):
        assert all(allowed[i] for i in t[n:])


def test_the_int8_target_is_near_the_one_in_16_bits():
    """The same weights: what codes of 8 bits lose. A value's code is off by half a step of a 127th of its row's largest; over K products
    of independent errors the logits are off by their norm times about sqrt(2) (0.5 / 127) (largest / rms) / sqrt(3): 3% a product at a
    largest of five times the rms, so under 10% after three."""
    import serve_drafts as ex
    plain, int8 = ex.Target(seed=1), ex.Target(seed=1, int8=True)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, 5, 512, generator=g).bfloat16().cuda()
    att = torch.randn(3, 5, 8, 64, generator=g).bfloat16().cuda()
    # the same network in double precision, with the norms that the 8-bit one has
    h = x.double() + (att.flatten(2) @ plain.o).double()
    norm = lambda t: t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    a, b = (norm(h) @ plain.up.double()).chunk(2, -1)
    want = norm(h + (torch.nn.functional.silu(a) * b) @ plain.down.double()) @ plain.head.double()
    got = int8.finish(x, att).double()
    assert (got - want).norm() <= 0.1 * want.norm()


def test_process_is_the_plain_form_over_the_text():
    import serve_drafts as ex
    text = [[5, 9, 9, 3], [7], [], [1, 2, 3, 1, 1]]
    prompts = [2, 1, 0, 5]
    g = torch.Generator().manual_seed(4)
    logits = torch.randn(4, 3, 64, generator=g).bfloat16()
    proposed = torch.randint(0, 64, (4, 2), generator=g, dtype=torch.int32)
    rates = dict(repetition=1.5, frequency=0.25, presence=0.5)
    got = ex.process(logits.cuda(), text, prompts, proposed.cuda(), rates, None).cpu().double()
    L = max(map(len, text))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    want, tol, _ = su.logits(logits, tokens=proposed, history=i32([t + [-1] * (L - len(t)) for t in text]), lengths=i32([len(t) for t in text]),
                             prompt=i32(prompts), **{k: torch.full((4,), v) for k, v in rates.items()})
    assert ((got - want).abs() <= tol + su.half_step(want, torch.bfloat16) * 1.01).all()


def test_one_product_workspace_serves_every_call():
    """Prompts, drafts and a table of the whole vocabulary, three weights: the one for the most tokens and the longest sums."""
    import serve_drafts as ex
    cache, target, text, _ = ex.serve(rounds=4, prompts=[9, 4, 17, 6], int8=True)
    assert len(target._product_ws) == 1 and all(sv.read_status(w) == 0 for w in target._product_ws.values())
    g = torch.Generator().manual_seed(5)
    ws, = target._product_ws.values()
    for tokens in (2048, 3, 700):
        x = torch.randn(1, tokens, 1024, generator=g).bfloat16().cuda()
        want = sv.int8_matmul(*sv.quantize_rows(x).values(), *target.int8["down"].values())["out"]
        assert torch.equal(target.product("down", sv.quantize_rows(x)), want)
    assert list(target._product_ws.values())[0] is ws
    target.product("up", sv.quantize_rows(torch.randn(1, 3000, 512, generator=g).bfloat16().cuda()))      # more than there were
    assert len(target._product_ws) == 1 and list(target._product_ws.values())[0].numel() > ws.numel()
