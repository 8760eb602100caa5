"""Borders of the operators between the last layer and a verification, on the GPU."""
import ctypes
import subprocess

import pytest
import torch

import score_util as su
import speculative_decoding_verification_target_gb300 as sv
from speculative_decoding_verification_target_gb300 import _build

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------------------------------- codes
def rows_of_codes(p):
    """Codes of fp32 values as they are and behind a norm, which takes the same ones."""
    got = sv.quantize_rows(p.cuda())["out"].cpu()
    assert torch.equal(sv.residual_norm(p.cuda(), quantize=True)["out"].cpu(), got)
    return got


@pytest.mark.parametrize("D", [768, 765, 9000])
def test_codes_next_to_the_middle_of_two(D):
    """m with all 24 bits, and the three values next to each (2 k + 1) m / 254: products that fp32 rounds decide. Rows of 16 bytes, value
    by value, and read twice."""
    odd = torch.arange(-253, 254, 2, dtype=torch.float64)
    rows = []
    for i, m in enumerate((1 + torch.rand(24, generator=gen(1))).tolist()):
        m = torch.tensor(m * 2.0 ** (i % 5 * 7 - 14), dtype=F32)
        p = (odd * m.double() / 254).float()
        near = torch.cat([p, torch.nextafter(p, m.expand(254)), torch.nextafter(p, -m.expand(254))])
        rows.append(torch.cat([m[None], near[:D - 1], torch.zeros(max(0, D - 1 - near.numel()))]))
    x = torch.stack(rows)
    codes, _ = su.exact_codes(x)
    assert torch.equal(rows_of_codes(x), codes)


@pytest.mark.parametrize("D", [256, 255, 8200])
def test_codes_on_the_middle_of_two(D):
    """m = 254 x and p = (2 k + 1) x, x of 16 bits: both 254 p and (2 k + 1) m are rounded, and equal all the same."""
    odd = torch.arange(-253, 254, 2, dtype=torch.float64)
    rows = []
    for x in (32769 + 2 * torch.randint(0, 16383, (24,), generator=gen(2))).tolist():
        row = torch.cat([torch.tensor([254.0], dtype=torch.float64), odd])[:D] * x
        assert torch.equal(row.float().double(), row)
        rows.append(torch.cat([row.float(), torch.zeros(max(0, D - 255))]))
    x = torch.stack(rows)
    codes, _ = su.exact_codes(x)
    assert torch.equal(rows_of_codes(x), codes)
    assert torch.equal(codes[0, 1:255] % 2, torch.zeros(min(D, 255) - 1, dtype=torch.int8))      # all ties go to the even one


@pytest.mark.parametrize("D", [256, 261, 16392, 16389])
def test_weighted_codes_on_the_middle_of_two(D):
    """fp16 rows times weights of 11 bits: p has 22 bits, and its ties are rounded products too. Rows of 16 bytes, rows that begin
    elsewhere, and rows that are read twice."""
    odd = torch.arange(-253, 254, 2, dtype=torch.float64)
    values = torch.cat([torch.tensor([254.0], dtype=torch.float64), odd])
    x = torch.stack([torch.cat([torch.zeros(s, dtype=torch.float64), values, torch.zeros(D, dtype=torch.float64)])[:D] * k for s, k in ((0, 5), (1, 7), (0, 3))])
    x = x.half()
    w = torch.full((D,), 2047 / 1024, dtype=F16)
    got = sv.residual_norm(x.cuda(), None, w.cuda(), quantize=True)["out"].cpu()
    codes, _ = su.exact_codes(x.float() * w.float())
    assert torch.equal(got, codes)


# ---------------------------------------------------------------------------------------- infinities and NaN
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("D", [261, 2051, 8193, 16385, 32768])
def test_infinities_and_nans_anywhere_in_a_row(D, dtype):
    """In a row's first and last values, and amid its pieces; every row of an odd width begins elsewhere."""
    places = (0, 1, 6, 7, 8, D // 2, D - 9, D - 8, D - 2, D - 1)
    n = len(places)
    x = torch.randn(2 * n, D, generator=gen(3)).to(dtype)
    res, w = torch.randn(2 * n, D, generator=gen(4)).to(dtype), (1 + 0.2 * torch.randn(D, generator=gen(5))).to(dtype)
    bad = x.clone()
    for i, at in enumerate(places):
        bad[2 * i, at] = (float("inf"), float("-inf"), float("nan"))[i % 3]
    fine = torch.arange(2 * n) % 2 == 1
    for r, weight in ((None, None), (res, w)):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        calls = [lambda v: sv.residual_norm(v.cuda(), c(r), c(weight), quantize=True)]
        if r is None:
            calls.append(lambda v: sv.quantize_rows(v.cuda()))
        for call in calls:
            want, got = call(x), call(bad)
            assert torch.isnan(got["scale"].cpu()[~fine]).all() and (got["out"].cpu()[~fine] == 0).all()
            for k in ("out", "scale"):
                assert torch.equal(got[k].cpu()[fine], want[k].cpu()[fine])
        want, got = (sv.residual_norm(v.cuda(), c(r), c(weight))["out"].cpu() for v in (x, bad))
        assert torch.equal(got[fine], want[fine]) and torch.isfinite(got[fine]).all()
        # with an infinity the row is infinitely long: 0 beside it, and NaN in its place; with a NaN all of it is
        for i, at in enumerate(places):
            row = got[2 * i]
            if i % 3 == 2:
                assert torch.isnan(row).all()
            else:
                rest = torch.cat([row[:at], row[at + 1:]])
                assert torch.isnan(row[at]) and (rest == 0).all()


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("rows,D", [(1217, 96), (700, 2048), (2000, 301), (1500, 2051), (400, 8192)])
def test_many_rows_of_other_types(rows, D, dtype):
    """Threads that take several rows one after the other."""
    x, res = (torch.randn(rows, D, generator=gen(s)).to(dtype) for s in (6, 7))
    w = (1 + 0.2 * torch.randn(D, generator=gen(8))).to(dtype)
    r, p, inv, v = su.norm(x, res, w, 1e-5)
    codes, s = su.exact_codes(p)
    got = sv.residual_norm(x.cuda(), res.cuda(), w.cuda(), 1e-5, quantize=True)
    assert torch.equal(got["residual"].cpu(), r) and torch.equal(got["out"].cpu(), codes)
    assert ((got["scale"].cpu().double() - s * inv).abs() <= su.inv_tol(D) * s * inv).all()
    got = sv.residual_norm(x.cuda(), res.cuda(), w.cuda(), 1e-5)
    assert torch.equal(got["residual"].cpu(), r)
    assert ((got["out"].cpu().double() - v).abs() <= su.half_step(v, dtype) * (1 + 2.0 ** -8) + su.inv_tol(D) * v.abs()).all()
    assert torch.equal(sv.quantize_rows(x.cuda())["out"].cpu(), su.exact_codes(x.float())[0])


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


LASTING = r"""
// lets the next kernel of its stream in and ends 2.5 s later, after 3000 naps at most
__global__ void lasting() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long from, now;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(from));
    for (int i = 0; i < 3000; ++i) {
        __nanosleep(1000000);
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
        if (now - from > 2500000000ull) break;
    }
}
extern "C" int last(void* stream) {
    lasting<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>();
    return cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def lasting(tmp_path_factory):
    d = tmp_path_factory.mktemp("lasting")
    (d / "lasting.cu").write_text(LASTING)
    subprocess.run([_build.nvcc_path(), "-gencode", "arch=compute_103a,code=sm_103a", "-Xcompiler", "-fPIC", "-shared", "-o", str(d / "lasting.so"),
                    str(d / "lasting.cu")], check=True)
    fn = ctypes.CDLL(str(d / "lasting.so")).last
    fn.argtypes = [ctypes.c_void_p]
    return fn


@pytest.mark.parametrize("M", [3, 16, 40, 300])
def test_a_kernel_in_front_may_last(M, lasting):
    """Longer than the two seconds after which a wait within the product gives up: those begin where that kernel ends."""
    g = gen(15)
    a, w = (torch.randint(-128, 128, (n, 1024), generator=g).to(torch.int8).cuda() for n in (M, 1024))
    sa, sw, ws = torch.ones(M, device="cuda"), torch.ones(1024, device="cuda"), sv.new_matmul_workspace(M, 1024, 1024)
    want = (a.double() @ w.double().t()).float()
    out = torch.empty(M, 1024, device="cuda")
    sv.int8_matmul(a, sa, w, sw, out=out, workspace=ws)      # loaded
    out.zero_()
    torch.cuda.synchronize()
    assert lasting(torch.cuda.current_stream().cuda_stream) == 0
    sv.int8_matmul(a, sa, w, sw, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert sv.read_status(ws) == 0 and torch.equal(out, want)


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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("masked", [False, True])
def test_as_many_listed_tokens_as_there_may_be(masked, dtype):
    """1024 tokens with a bias and 64 others among the drafts, all in one part of the vocabulary; enough sequences that it is one."""
    B, R, V, n = 608, 65, 1500, 1024
    g = gen(13)
    order = torch.randperm(V, generator=g).int()
    x = torch.randn(B, R, V, device="cuda", generator=torch.Generator("cuda").manual_seed(14)).to(dtype)
    a = dict(tokens=order[n:n + R - 1].expand(B, -1).contiguous(), bias_tokens=order[:n].expand(B, -1).contiguous(),
             bias=4 * torch.randn(B, n, generator=g), history=torch.randint(0, V, (B, 40), generator=g, dtype=torch.int32),
             lengths=torch.full((B,), 40, dtype=torch.int32), prompt=torch.full((B,), 13, dtype=torch.int32),
             repetition=1 + torch.rand(B, generator=g), frequency=torch.rand(B, generator=g), presence=torch.rand(B, generator=g))
    if masked:
        a["mask"] = torch.randint(-2 ** 31, 2 ** 31, (1, R, (V + 31) // 32), generator=g).int().expand(B, -1, -1)
    got = sv.process_logits(x, **{k: v.cuda() for k, v in a.items()})["out"]
    for b in (0, 303, B - 1):
        want, tol, same = su.logits(x[b:b + 1].cpu(), **{k: v[b:b + 1] for k, v in a.items()})
        out, fine = got[b:b + 1].cpu(), torch.isfinite(want)
        assert torch.equal(out[same], x[b:b + 1].cpu()[same]) and torch.equal(torch.isfinite(out), fine)
        assert ((out.double() - want).abs() <= tol + su.half_step(want, dtype) * (1 + 2.0 ** -8))[fine].all()
