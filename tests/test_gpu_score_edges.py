"""Borders of the operators between the last layer and a verification, on the GPU."""
import pytest
import torch

import speculative_decoding_verification_target_gb300 as sv

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


# ----------------------------------------------------------------------------------------------------- product
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("C,K", [(257, 512), (300, 4096), (200, 301)])
def test_a_bias_is_added_to_the_rounded_product_whatever_the_tokens(C, K, dtype):
    """Bit for bit, and the same for a token alone, among few and among many."""
    g = gen(9)
    M = 150
    a = (32 * torch.randn(M, K, generator=g)).round().clamp(-127, 127).to(torch.int8)
    w = torch.randint(-128, 128, (C, K), generator=g).to(torch.int8)
    sa, sw = 0.01 + torch.rand(M, generator=g), 0.01 + torch.rand(C, generator=g)
    total = (a.double() @ w.double().t()).float()
    bias = total[3] * sa[3] * sw * (torch.rand(C, generator=g) - 1.2)      # much of what they are added to is taken off again
    want = (total * (sa[:, None] * sw) + bias).to(dtype)
    for n in (1, 2, 4, 7, 8, 9, 20, 33, 70, M):
        got = sv.int8_matmul(a[:n].cuda(), sa[:n].cuda(), w.cuda(), sw.cuda(), bias=bias.cuda(), dtype=dtype)["out"]
        assert torch.equal(got.cpu(), want[:n]), n


# ------------------------------------------------------------------------------------------------------ logits
@pytest.mark.parametrize("V", [1000, 1003])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_repetition_divides(V, dtype):
    """y / repetition as fp32 rounds it, for tokens of the history and, listed, for drafts and those with a bias."""
    reps = torch.tensor([1.1, 1.3, 3.0, 0.7, 7.0, 1e-3, 2.5e38, 1.5])
    B, R = reps.numel(), 3
    x = (5 * torch.randn(B, R, V, generator=gen(10))).to(dtype)
    history = torch.arange(V, dtype=torch.int32).expand(B, V).contiguous()
    lengths = torch.full((B,), V // 2, dtype=torch.int32)
    prompt = torch.tensor([V, 0] * (B // 2), dtype=torch.int32)      # all asked, or all said
    tokens = torch.stack([torch.randperm(V, generator=gen(11))[:R - 1] for _ in range(B)]).int()
    ids = torch.arange(0, V, 9, dtype=torch.int32).expand(B, -1).contiguous()
    add = torch.randn(B, ids.shape[1], generator=gen(12))
    got = sv.process_logits(x.cuda(), tokens=tokens.cuda(), history=history.cuda(), lengths=lengths.cuda(), prompt=prompt.cuda(),
                            repetition=reps.cuda(), bias_tokens=ids.cuda(), bias=add.cuda())["out"].cpu()
    y = x.float().clone()
    y[:, :, ids[0].long()] += add[:, None]
    seen = torch.zeros(B, R, V, dtype=torch.bool)
    seen[:, :, :V // 2] = True
    for b in range(B):
        for j in range(1, R):
            seen[b, j:, int(tokens[b, j - 1])] = True
    rep = reps[:, None, None]
    want = torch.where(seen, torch.where(y > 0, y / rep, y * rep), y)
    assert torch.equal(got, want.to(dtype))
