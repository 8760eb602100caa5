"""The operators between the last layer and a verification on the GPU, against plain forms in 64 bits (score_util)."""
import pytest
import torch

import score_util as su
import speculative_decoding_verification_target_gb300 as sv

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, F16, F32]


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def values(rows, D, dtype, seed, scale=1.0):
    g = gen(seed)
    return (scale * torch.randn(rows, D, generator=g) * torch.exp(0.7 * torch.randn(D, generator=g))).to(dtype)


# --------------------------------------------------------------------------------------------- norm and codes
def check_norm(x, residual, weight, eps, quantize, **kw):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = sv.residual_norm(dev(x), dev(residual), dev(weight), eps, quantize=quantize, **kw)
    r, p, inv, v = su.norm(x, residual, weight, eps)
    D = x.shape[1]
    if residual is not None:
        assert torch.equal(got["residual"].cpu(), r)
    if quantize:
        codes, s = su.exact_codes(p)
        assert torch.equal(got["out"].cpu(), codes)
        want = s * inv
        assert ((got["scale"].cpu().double() - want).abs() <= su.inv_tol(D) * want + 1e-45).all()
    else:
        assert got["scale"] is None
        tol = su.half_step(v, x.dtype) * (1 + 2.0 ** -8) + su.inv_tol(D) * v.abs()
        assert ((got["out"].cpu().double() - v).abs() <= tol).all()


WIDTHS = [1, 2, 7, 8, 31, 32, 33, 64, 127, 128, 255, 256, 257, 261, 263, 511, 1000, 1024, 2050, 2051, 4095, 4096, 4097, 4104, 8192, 10007, 16383, 16384, 16385, 32760, 32768]


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_norm(D, dtype, quantize):
    for rows, residual, weight, seed in ((3, True, True, 1), (1, False, True, 2), (5, True, False, 3), (2, False, False, 4)):
        check_norm(values(rows, D, dtype, seed), values(rows, D, dtype, seed + 10, 3.0) if residual else None,
                   (1 + 0.2 * torch.randn(D, generator=gen(seed + 20))).to(dtype) if weight else None, 1e-6, quantize)


@pytest.mark.parametrize("rows,D", [(1, 4096), (6, 4096), (151, 512), (1217, 96), (700, 2048), (3001, 264), (400, 8192), (1500, 2051), (700, 4099), (2000, 301)])
def test_norm_of_many_rows(rows, D):
    x, res, w = values(rows, D, BF16, 5), values(rows, D, BF16, 6, 3.0), (1 + 0.2 * torch.randn(D, generator=gen(7))).bfloat16()
    for quantize in (False, True):
        check_norm(x, res, w, 1e-5, quantize)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1, 5, 64, 1023, 4096, 14336])
def test_quantize_rows(D, dtype):
    x = values(9, D, dtype, 8, 0.1)
    x[3] = 0
    got = sv.quantize_rows(x.cuda())
    codes, s = su.exact_codes(x.float())
    assert torch.equal(got["out"].cpu(), codes)
    # m / 127 rounded once, or by a product with a rounded 1 / 127: two half steps
    assert ((got["scale"].cpu().double() - s).abs() <= 2 * 2.0 ** -24 * s + 1e-45).all()
    assert float(got["scale"][3]) == 0.0


@pytest.mark.parametrize("dtype", TYPES)
def test_codes_at_the_borders(dtype):
    """Values that lie on the middle between two codes, and the neighbours of those: 127 p / m = k + 1/2 for m = 254 and 127."""
    half = torch.arange(-126.5, 127, 1.0)
    rows = []
    for m, step in ((254.0, 2.0), (127.0, 1.0)):
        p = (half * step).to(dtype)
        up = (p.float() * (1 + torch.finfo(dtype).eps)).to(dtype)
        down = (p.float() * (1 - torch.finfo(dtype).eps)).to(dtype)
        rows += [torch.cat([torch.tensor([m], dtype=dtype), q]) for q in (p, up, down)]
    for scale in (1.0, 2.0 ** -10, 2.0 ** 7):
        x = torch.stack(rows) * scale
        codes, _ = su.exact_codes(x.float())
        assert torch.equal(sv.quantize_rows(x.cuda())["out"].cpu(), codes)
    if dtype is not F16:      # far from 1, where a reciprocal or the products would leave fp32's range
        for scale in (2.0 ** -133, 2.0 ** -120, 2.0 ** 110):
            x = torch.stack(rows) * torch.tensor(scale, dtype=dtype)
            codes, _ = su.exact_codes(x.float())
            assert torch.equal(sv.quantize_rows(x.cuda())["out"].cpu(), codes)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [40, 33])
def test_rows_with_infinities_and_nans(D, dtype):
    x = values(6, D, dtype, 9)
    x[0, 3], x[1, 0], x[2, -1], x[3, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    x[3, 2] = float("inf")
    want = sv.quantize_rows(x[4:].cuda())
    for got in (sv.quantize_rows(x.cuda()), sv.residual_norm(x.cuda(), quantize=True)):
        assert torch.isnan(got["scale"][:4]).all() and torch.isfinite(got["scale"][4:]).all()
        assert (got["out"][:4] == 0).all() and torch.equal(got["out"][4:], want["out"])
    out = sv.residual_norm(x.cuda())["out"]
    assert torch.isfinite(out[4:]).all() and torch.isnan(out[1]).all() and torch.isnan(out[3]).all()


def test_norm_of_zeros():
    z = torch.zeros(2, 96, dtype=BF16, device="cuda")
    got = sv.residual_norm(z, z, quantize=True, eps=0.0)
    assert (got["out"] == 0).all() and (got["residual"] == 0).all()
    got = sv.residual_norm(z, z, quantize=True)
    assert (got["out"] == 0).all() and (got["scale"] == 0).all()


@pytest.mark.parametrize("D", [1024, 20000])
def test_norm_in_both_inputs_places(D):
    """out in x's place and the residual in its own, and the other way round; a weight that does not begin on 16 bytes; repeated rows."""
    x, res, buf = values(40, D, BF16, 70).cuda(), values(40, D, BF16, 71, 3.0).cuda(), torch.rand(D + 3, generator=gen(72)).bfloat16().cuda()
    w = buf[3:]
    want = sv.residual_norm(x, res, w)
    check_norm(x.cpu(), res.cpu(), w.cpu(), 1e-6, False)
    for swap in (False, True):
        a, b = x.clone(), res.clone()
        sv.residual_norm(a, b, w, out=b if swap else a, residual_out=a if swap else b)
        assert torch.equal(b if swap else a, want["out"]) and torch.equal(a if swap else b, want["residual"])
    got = sv.residual_norm(x[:1].expand(7, D), res[:1].expand(7, D), w)
    assert torch.equal(got["out"], want["out"][:1].expand(7, D)) and torch.equal(got["residual"], want["residual"][:1].expand(7, D))


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("D", [512, 520, 509])
def test_norm_strides_places_and_shapes(D, quantize):
    """Rows of a wider buffer, transposed leading dimensions, an odd start, [B, N, D], and outputs in the inputs' places."""
    B, N = 3, 5
    full = values(B * N, D, BF16, 11)
    res, w = values(B * N, D, BF16, 12, 3.0), torch.ones(D).bfloat16()
    plain = sv.residual_norm(full.cuda(), res.cuda(), w.cuda(), quantize=quantize)
    for off, pad in ((0, 8), (1, 0), (8, 3)):
        buf = torch.full((N, B, D + off + pad), 7.0, dtype=BF16, device="cuda")
        x = buf[:, :, off:off + D].transpose(0, 1)
        x.copy_(full.view(B, N, D))
        before = buf.clone()
        got = sv.residual_norm(x, res.cuda().view(B, N, D), w.cuda(), quantize=quantize)
        for k in ("out", "residual"):
            assert torch.equal(got[k].view(B * N, D), plain[k])
        assert torch.equal(buf, before)
        r = res.cuda().view(B, N, D).clone()
        out = None if quantize else x
        got = sv.residual_norm(x, r, w.cuda(), quantize=quantize, residual_out=r, out=out)
        assert got["residual"] is r and torch.equal(r.view(B * N, D), plain["residual"])
        assert torch.equal(got["out"].reshape(B * N, D), plain["out"])
        rim = torch.ones_like(buf, dtype=torch.bool)
        rim[:, :, off:off + D] = False
        assert torch.equal(buf[rim], before[rim])
    if quantize:
        assert torch.equal(sv.residual_norm(full.cuda().view(B, N, D), res.cuda().view(B, N, D), w.cuda(), quantize=True)["scale"],
                           plain["scale"].view(B, N))
        wide = torch.full((B * N, D + 3), 77, dtype=torch.int8, device="cuda")
        sv.residual_norm(full.cuda(), res.cuda(), w.cuda(), quantize=True, out=wide[:, 2:2 + D])
        assert torch.equal(wide[:, 2:2 + D], plain["out"]) and (wide[:, :2] == 77).all() and (wide[:, 2 + D:] == 77).all()


# ------------------------------------------------------------------------------------------------- product
def ints(rows, K, seed, kind="normal"):
    g = gen(seed)
    if kind == "normal":
        return (32 * torch.randn(rows, K, generator=g)).round().clamp(-127, 127).to(torch.int8)
    if kind == "any":
        return torch.randint(-128, 128, (rows, K), generator=g).to(torch.int8)
    return torch.full((rows, K), {"top": 127, "bottom": -128}[kind], dtype=torch.int8)


def check_product(a, w, seed=0, dtype=BF16, bias=False, **kw):
    """Without a bias bit for bit: fp32 of the exact sum, times the rounded product of the scales, rounded."""
    M, C = a.shape[0], w.shape[0]
    g = gen(seed)
    sa, sw = 0.01 + torch.rand(M, generator=g), 0.01 + torch.rand(C, generator=g)
    b = 100 * torch.randn(C, generator=g) if bias else None
    got = sv.int8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), bias=None if b is None else b.cuda(), dtype=dtype, **kw)
    assert sv.read_status(got["workspace"]) == 0
    total = (a.cuda().double() @ w.cuda().double().t()).cpu()
    y = total.float() * (sa[:, None] * sw)
    if not bias:
        assert torch.equal(got["out"].cpu(), y.to(dtype))
    else:      # the product and its sum with the bias are rounded once or twice in fp32, then to dtype
        want = total * (sa[:, None] * sw).double() + b.double()
        fp32 = 2.0 ** -23 * (y.abs().double() + b.abs().double())
        tol = fp32 + su.half_step(want, dtype) * (1 + 2.0 ** -8)
        out = got["out"].cpu().double()
        # fp16 ends at 65504 with a step of 32: from 65520 on a value rounds to infinity
        top = 65520 if dtype is F16 else torch.inf
        over = torch.isinf(out)
        assert (want.abs() + fp32 >= top)[over].all() and (out.sign() == want.sign())[over].all()
        assert ((out - want).abs() <= tol)[~over].all() and (want.abs() - fp32 < top)[~over].all()


SHAPES = [(1, 1, 1), (1, 1, 16), (1, 128, 64), (2, 3, 4), (1, 4096, 4096), (3, 129, 512), (7, 127, 1000), (8, 256, 528), (16, 128, 128),
          (17, 300, 144), (33, 1000, 2064), (64, 512, 513), (65, 64, 4096), (96, 640, 1024), (129, 257, 112), (192, 256, 1536),
          (193, 384, 640), (200, 130, 48), (256, 1024, 4096), (384, 2000, 1040), (385, 515, 16), (1000, 768, 272), (1, 70, 16400),
          (5, 40, 131071), (2, 16, 131056), (640, 33, 2048), (65, 9800, 272), (70, 38900, 144), (193, 6000, 400), (250, 5001, 2064),
          (1000, 2100, 640), (2500, 1300, 128), (9, 20000, 64), (40, 5000, 16400), (100, 300, 4097), (40, 129, 16399), (513, 1000, 1001), (130, 5, 5000), (4, 20000, 4096),
          (3, 12000, 4096), (4, 16, 1000), (300, 9999, 130), (9, 5000, 128), (31, 30000, 384), (32, 129, 4112), (17, 40000, 640),
          (24, 1000, 96)]


@pytest.mark.parametrize("M,C,K", SHAPES)
def test_product(M, C, K):
    check_product(ints(M, K, 1), ints(C, K, 2, "any"), 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias", [False, True])
def test_product_types(dtype, bias):
    for M, C, K in ((5, 200, 256), (70, 513, 1024), (6, 31, 77)):
        check_product(ints(M, K, 4), ints(C, K, 5), 6, dtype, bias)


@pytest.mark.parametrize("K", [16, 1024, 1040, 16384, 131056, 999])
def test_sums_are_exact_at_their_largest(K):
    """All products of one sign and at their largest, alone and with odd ones among them: sums that fp32 could not hold."""
    for ka, kw in (("bottom", "bottom"), ("top", "top"), ("top", "bottom")):
        check_product(ints(20, K, 0, ka), ints(150, K, 0, kw), 7, F32)
        a = ints(20, K, 0, ka)
        a[:, ::7] = ints(20, K, 8, "any")[:, ::7]
        check_product(a, ints(150, K, 0, kw), 7, F32)


def test_product_strides_and_rims():
    """Operands and outputs in wider buffers, [B, N, K], outputs in their place and nothing beside them."""
    B, N, C, K = 3, 7, 200, 320
    a, w = ints(B * N, K, 9), ints(C, K, 10)
    sa, sw = (0.1 + torch.rand(n, generator=gen(11)) for n in (B * N, C))
    plain = sv.int8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda())["out"]
    for pa, pw, off in ((0, 0, 0), (16, 32, 16), (5, 16, 0), (16, 3, 16), (1, 1, 1)):
        ba = torch.full((N, B, K + pa + off), 99, dtype=torch.int8, device="cuda")
        bw = torch.full((C, K + pw + off), 99, dtype=torch.int8, device="cuda")
        av, wv = ba[:, :, off:off + K].transpose(0, 1), bw[:, off:off + K]
        av.copy_(a.view(B, N, K))
        wv.copy_(w)
        buf = torch.full((B, N, C + 9), 5.0, dtype=BF16, device="cuda")
        got = sv.int8_matmul(av, sa.cuda().view(B, N), wv, sw.cuda(), out=buf[:, :, 4:4 + C])["out"]
        assert torch.equal(got.reshape(B * N, C), plain)
        assert (buf[:, :, :4] == 5).all() and (buf[:, :, 4 + C:] == 5).all()


@pytest.mark.parametrize("M", [1, 5, 40])
def test_product_of_rows_that_repeat_or_overlap(M):
    """Inputs may: one token's codes for all, one channel's for all, and channels that begin 16 or 5 codes after one another."""
    K, C = 320, 70
    one, long = ints(1, K, 50).cuda(), ints(1, K + 16 * C, 51, "any").cuda()[0]
    sa, sw = torch.ones(M, device="cuda"), torch.ones(C, device="cuda")
    for a in (ints(M, K, 52).cuda(), one.expand(M, K)):
        for w in (one.expand(C, K), long.as_strided((C, K), (16, 1)), long.as_strided((C, K), (5, 1), 3)):
            got = sv.int8_matmul(a, sa, w, sw, dtype=F32)["out"]
            assert torch.equal(got.double(), a.double() @ w.double().t())


def test_a_workspace_that_is_not_given_is_ready():
    """Also one so large that only its header is cleared."""
    a, w = ints(600, 1024, 53).cuda(), ints(300, 1024, 54).cuda()
    torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")      # what the allocator may hand out
    r = sv.int8_matmul(a, torch.ones(600, device="cuda"), w, torch.ones(300, device="cuda"), dtype=F32)
    assert r["workspace"].numel() > 1 << 16 and sv.read_status(r["workspace"]) == 0
    assert torch.equal(r["out"].double(), a.double() @ w.double().t())


def test_a_scale_of_nan_stays_in_its_row():
    a, w = ints(40, 256, 12), ints(100, 256, 13)
    sa, sw = torch.ones(40), torch.ones(100)
    sa[3], sw[5] = float("nan"), float("inf")
    out = sv.int8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), dtype=F32)["out"].cpu()
    assert torch.isnan(out[3]).all() and torch.equal(torch.isfinite(out[0]), sw.isfinite())


def test_one_workspace_serves_smaller_calls():
    ws = sv.new_matmul_workspace(400, 3000, 2048)
    for M, C, K in ((400, 3000, 2048), (1, 3000, 2048), (400, 5, 2048), (33, 700, 64), (3, 2999, 2000), (200, 1000, 1008)):
        check_product(ints(M, K, 14), ints(C, K, 15), 16, workspace=ws)


# ------------------------------------------------------------------------------------------------- logits
def check_logits(B, R, V, dtype=BF16, L=50, biases=0, mask=None, seed=0, **drop):
    g = gen(seed)
    a = dict(x=(3 * torch.randn(B, R, V, generator=g)).to(dtype), tokens=torch.randint(0, V, (B, R), generator=g, dtype=torch.int32),
             history=(torch.rand(B, L, generator=g) ** 2 * V).int(), lengths=torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32),
             repetition=1 + torch.rand(B, generator=g), frequency=torch.rand(B, generator=g), presence=torch.rand(B, generator=g))
    a["lengths"][0] = L
    a["prompt"] = (a["lengths"] * torch.rand(B, generator=g)).int()
    if biases:
        a["bias_tokens"] = torch.randint(-1, V, (B, biases), generator=g, dtype=torch.int32)
        a["bias"] = 5 * torch.randn(B, biases, generator=g)
    if mask:
        W = (V + 31) // 32
        words = torch.randint(-2 ** 31, 2 ** 31, (B, R, W), generator=g)
        a["mask"] = {"any": words, "none": torch.zeros_like(words), "all": torch.full_like(words, -1)}[mask].int()
    a.update(drop)
    run_logits(a)


def run_logits(a, **kw):
    x = a["x"]
    rest = {k: v for k, v in a.items() if k != "x" and v is not None}
    got = sv.process_logits(x.cuda(), **{k: v.cuda() for k, v in rest.items()}, **kw)["out"].cpu()
    want, tol, same = su.logits(x, **rest)
    kind = torch.int16 if x.dtype is BF16 else torch.int32
    assert torch.equal(got.view(kind)[same], x.view(kind)[same])
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)].double(), want[~fine & ~torch.isnan(want)])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert ((got.double() - want).abs() <= tol + su.half_step(want, x.dtype) * (1 + 2.0 ** -8))[fine].all()


VOCABULARIES = [1, 2, 31, 32, 33, 63, 100, 1000, 1001, 2047, 2048, 8191, 8192, 8193, 16384, 16400, 32001]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", VOCABULARIES)
def test_logits(V, dtype):
    check_logits(2, 4, V, dtype, biases=6, mask="any", seed=V)
    check_logits(3, 1, V, dtype, L=300, seed=V + 1)


@pytest.mark.parametrize("B,R,V,L", [(1, 1, 128256, 2000), (1, 65, 1000, 10), (5, 21, 4099, 700), (2, 6, 151936, 3000), (70, 2, 500, 1),
                                     (1, 2, 262144, 5000), (1, 3, 50257, 40000)])
def test_logits_sizes(B, R, V, L):
    check_logits(B, R, V, L=L, biases=5, seed=1)


@pytest.mark.parametrize("left_out", ["tokens", "history", "prompt", "repetition", "frequency", "presence", "mask", "bias_tokens"])
def test_parts_left_out(left_out):
    drop = {left_out: None}
    if left_out == "history":
        drop.update(lengths=None, prompt=None)
    if left_out == "bias_tokens":
        drop.update(bias=None)
    check_logits(3, 4, 777, biases=9, seed=3, **{"mask": "any", **drop})


def test_nothing_asked_for_is_a_copy():
    x = torch.randn(2, 3, 1003, device="cuda").bfloat16()
    x[0, 0, :3] = torch.tensor([float("nan"), float("inf"), float("-inf")])
    got = sv.process_logits(x)["out"]
    assert torch.equal(got.view(torch.int16), x.view(torch.int16)) and got.data_ptr() != x.data_ptr()


@pytest.mark.parametrize("kind", ["none", "all"])
@pytest.mark.parametrize("V", [32, 1000, 9001])
def test_masks_of_everything_and_nothing(kind, V):
    check_logits(2, 3, V, mask=kind, seed=4)


def test_masked_places_hold_anything():
    """Infinities and NaN under a mask are -inf; where they are allowed they follow the arithmetic."""
    x = torch.zeros(1, 1, 64)
    x[0, 0, :8] = torch.tensor([float("nan"), float("inf"), float("-inf"), 3.0, float("nan"), float("inf"), float("-inf"), -3.0])
    mask = torch.tensor([[[0xF0, -1]]], dtype=torch.int32)
    h = torch.arange(8, dtype=torch.int32)[None]
    a = dict(x=x, history=h, lengths=torch.tensor([8], dtype=torch.int32), mask=mask, repetition=torch.tensor([2.0]),
             frequency=torch.tensor([1.0]))
    run_logits(a)
    got = sv.process_logits(**{("logits" if k == "x" else k): v.cuda() for k, v in a.items()})["out"][0, 0, :8].cpu()
    assert (got[:4] == -torch.inf).all() and torch.isnan(got[4]) and got[5] == torch.inf and got[6] == -torch.inf and got[7] == -7.0


def test_ids_outside_the_vocabulary_are_passed_over():
    V = 500
    bad = torch.tensor([[-1, V, 2 ** 31 - 1, -2 ** 31, V + 1, -8192, 17, 8192, 3]], dtype=torch.int32)
    one = torch.ones(1)
    x = torch.randn(1, 4, V, generator=gen(5))
    run_logits(dict(x=x, history=bad, lengths=torch.tensor([9], dtype=torch.int32), prompt=torch.tensor([5], dtype=torch.int32),
                    tokens=torch.tensor([[V, -1, -2 ** 31]], dtype=torch.int32), repetition=2 * one, frequency=one, presence=one,
                    bias_tokens=bad, bias=torch.arange(9.0)[None]))


def test_lengths_and_prompts_outside_the_history():
    x = torch.randn(4, 2, 300, generator=gen(6))
    h = torch.randint(0, 300, (4, 20), generator=gen(7), dtype=torch.int32)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    run_logits(dict(x=x, history=h, lengths=i32(-5, 0, 21, 2 ** 31 - 1), prompt=i32(-1, 5, 100, -2 ** 31), frequency=torch.ones(4),
                    repetition=torch.full((4,), 1.5)))


def test_untouched_logits_keep_their_values():
    """Next to penalised tokens: infinities, NaN, zeros of both signs and subnormal numbers, in place too."""
    for dtype in (BF16, F32):
        x = torch.randn(1, 2, 64, generator=gen(60)).to(dtype)
        x[0, :, 1:8] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0, 0.0, 1e-40, -1e-39]).to(dtype)
        h = torch.arange(0, 64, 8, dtype=torch.int32)[None].cuda()
        a = dict(history=h, lengths=torch.tensor([8], dtype=torch.int32).cuda(), repetition=torch.tensor([1.5]).cuda(),
                 frequency=torch.tensor([0.5]).cuda(), bias_tokens=torch.tensor([[9]], dtype=torch.int32).cuda(), bias=torch.tensor([[2.0]]).cuda())
        y = x.cuda()
        for got in (sv.process_logits(x.cuda(), **a)["out"], sv.process_logits(y, out=y, **a)["out"]):
            for i in list(range(1, 8)) + list(range(10, 16)):
                p, q = got[0, :, i].cpu(), x[0, :, i]
                assert torch.equal(torch.isnan(p), torch.isnan(q)) and torch.equal(torch.signbit(p[~torch.isnan(p)]), torch.signbit(q[~torch.isnan(q)]))
                assert torch.equal(p[~torch.isnan(p)], q[~torch.isnan(q)])
            assert torch.equal(got[0, :, 9].cpu(), (x[0, :, 9].float() + 2).to(dtype))


def test_repeated_entries():
    """The same token over and over: in the history (counted), among the drafts, and among the biases (the last counts)."""
    V = 9000
    h = torch.full((1, 70000), 8200, dtype=torch.int32)
    h[0, ::2] = 3
    run_logits(dict(x=torch.randn(1, 5, V, generator=gen(8)), history=h, lengths=torch.tensor([70000], dtype=torch.int32),
                    prompt=torch.tensor([1001], dtype=torch.int32), tokens=torch.full((1, 4), 3, dtype=torch.int32),
                    frequency=torch.tensor([0.25]), presence=torch.tensor([0.5]), repetition=torch.tensor([1.25]),
                    bias_tokens=torch.tensor([[3, 3, 8200, 3, 8200]], dtype=torch.int32),
                    bias=torch.tensor([[1.0, 2.0, 4.0, -8.0, 16.0]])))


@pytest.mark.parametrize("V", [1000, 1001, 8200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logits_strides_masks_for_several_rows_and_in_place(V, dtype):
    B, R = 2, 3
    g = gen(9)
    x = torch.randn(B, R, V, generator=g).to(dtype)
    one = torch.randint(-2 ** 31, 2 ** 31, (B, 1, (V + 31) // 32), generator=g).int()
    a = dict(history=torch.randint(0, V, (B, 30), generator=g, dtype=torch.int32).cuda(), lengths=torch.full((B,), 30, dtype=torch.int32).cuda(),
             repetition=torch.full((B,), 1.3).cuda(), tokens=torch.randint(0, V, (B, R - 1), generator=g, dtype=torch.int32).cuda())
    plain = sv.process_logits(x.cuda(), mask=one.expand(B, R, -1).contiguous().cuda(), **a)["out"]
    mask = one.cuda().expand(B, R, -1)
    assert torch.equal(sv.process_logits(x.cuda(), mask=mask, **a)["out"], plain)
    for off, pad in ((0, 8), (1, 0), (3, 5)):
        buf = torch.full((R, B, V + off + pad), 7.0, dtype=dtype, device="cuda")
        view = buf[:, :, off:off + V].transpose(0, 1)
        view.copy_(x)
        assert torch.equal(sv.process_logits(view, mask=mask, **a)["out"], plain)
        out = torch.full((B, R, V + 4), 6.0, dtype=dtype, device="cuda")
        sv.process_logits(view, mask=mask, out=out[:, :, 1:1 + V], **a)
        assert torch.equal(out[:, :, 1:1 + V], plain) and (out[:, :, :1] == 6).all() and (out[:, :, 1 + V:] == 6).all()
        got = sv.process_logits(view, mask=mask, out=view, **a)["out"]
        assert got is view and torch.equal(view, plain)
        rim = torch.ones_like(buf, dtype=torch.bool)
        rim[:, :, off:off + V] = False
        assert (buf[rim] == 7).all()


# ----------------------------------------------------------------------------------- together, streams, graphs
def chain(x, residual, weight, codes, scale, logits_args, ws, tokens, draft, seeds, **kw):
    r = sv.residual_norm(x, residual, weight, quantize=True, **kw)
    y = sv.int8_matmul(r["out"], r["scale"], codes, scale, workspace=ws, **kw)["out"]
    z = sv.process_logits(y, tokens=tokens, out=y, **logits_args, **kw)["out"]
    d = sv.process_logits(draft, tokens=tokens, **{**logits_args, "mask": None}, **kw)["out"]
    return z, d, sv.verify(z, d, tokens, seeds, 1.0, **kw)


def chain_inputs(B=4, K=3, V=1000, D=512, seed=0):
    g = gen(seed)
    c = lambda t: t.cuda()  # noqa: E731
    x, res = (torch.randn(B, K + 1, D, generator=g).bfloat16() for _ in range(2))
    head = sv.quantize_rows(c(0.2 * torch.randn(V, D, generator=g).bfloat16()))
    tokens = c(torch.randint(0, V, (B, K), generator=g, dtype=torch.int32))
    mask = torch.randint(-2 ** 31, 2 ** 31, (B, K + 1, (V + 31) // 32), generator=g).int()
    args = dict(history=c(torch.randint(0, V, (B, 64), generator=g, dtype=torch.int32)), lengths=c(torch.tensor([64, 0, 5, 33], dtype=torch.int32)),
                prompt=c(torch.tensor([20, 0, 5, 1], dtype=torch.int32)), repetition=c(1 + torch.rand(B, generator=g)),
                frequency=c(torch.rand(B, generator=g)), mask=c(mask))
    draft = c(torch.randn(B, K, V, generator=g).bfloat16())
    return dict(x=c(x), residual=c(res), weight=torch.ones(D, device="cuda").bfloat16(), codes=head["out"], scale=head["scale"],
                logits_args=args, ws=sv.new_matmul_workspace(B * (K + 1), V, D), tokens=tokens, draft=draft,
                seeds=torch.arange(B, dtype=torch.int64, device="cuda"))


def test_a_chain_of_calls_into_a_verification():
    """Norm, product, penalties and mask, verification, each step against its plain form from the step before; the verification
    accepts no token that the mask forbids."""
    a = chain_inputs()
    z, d, v = chain(**a)
    B, R, V = z.shape
    r, p, inv, _ = su.norm(a["x"].cpu().flatten(0, 1), a["residual"].cpu().flatten(0, 1), None, 1e-6)
    codes, s = su.exact_codes(p)
    total = codes.double() @ a["codes"].cpu().double().t()
    y = (total * (s * inv)[:, None] * a["scale"].cpu().double()).view(B, R, V)
    rest = {k: t.cpu() for k, t in a["logits_args"].items()}
    want, tol, _ = su.logits(y, tokens=a["tokens"].cpu(), **rest)
    rep = rest["repetition"][:, None, None].double()
    # the product's bf16 rounding (half a step of 2^-8, stretched by the penalty) and the result's
    tol = tol + (su.half_step(y, BF16) + 1e-4 * y.abs()) * rep + su.half_step(want, BF16) * 1.01
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(z.cpu())) and ((z.cpu().double() - want).abs() <= tol)[fine].all()
    allowed = torch.isfinite(want)
    for b, (n, toks) in enumerate(zip(v["accept_len"].tolist(), v["out_tokens"].tolist())):
        assert all(allowed[b, j, t] for j, t in enumerate(toks[:n + 1]))


def test_on_another_stream_and_captured():
    a = chain_inputs(seed=1)
    z, d, v = chain(**a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z2, d2, v2 = chain(**a, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in ((z, z2), (d, d2), (v["out_tokens"], v2["out_tokens"])):
        assert torch.equal(p, q)
    fixed = {k: t.clone() for k, t in a.items() if torch.is_tensor(t)}
    fixed.update(logits_args=a["logits_args"], ws=sv.new_matmul_workspace(16, 1000, 512))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z3, d3, v3 = chain(**fixed)
    b = chain_inputs(seed=2)
    want = chain(**{**b, "codes": a["codes"], "scale": a["scale"], "logits_args": a["logits_args"]})
    for k in ("x", "residual", "tokens", "draft", "seeds"):
        fixed[k].copy_(b[k])
    for _ in range(3):
        graph.replay()
        assert torch.equal(z3, want[0]) and torch.equal(d3, want[1]) and torch.equal(v3["out_tokens"], want[2]["out_tokens"])


def test_two_products_at_once_on_two_streams():
    """Each with its own workspace, many times over."""
    jobs = []
    for i, (M, C, K) in enumerate(((50, 4000, 2048), (300, 1500, 1024))):
        a, w = ints(M, K, 20 + i).cuda(), ints(C, K, 30 + i).cuda()
        one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
        jobs.append((a, one(M), w, one(C), sv.new_matmul_workspace(M, C, K), torch.cuda.Stream(), (a.double() @ w.double().t()).float()))
    torch.cuda.synchronize()
    outs = [[sv.int8_matmul(a, sa, w, sw, dtype=F32, workspace=ws, stream=s)["out"] for a, sa, w, sw, ws, s, _ in jobs] for _ in range(20)]
    torch.cuda.synchronize()
    for row in outs:
        for got, job in zip(row, jobs):
            assert torch.equal(got, job[-1])


@pytest.mark.parametrize("M,C,K", [(1100, 11, 2048), (4265, 11, 13648), (300, 40, 1024), (12, 700, 4096), (384, 9999, 512), (200, 900, 3999), (30, 25000, 1152), (20, 400, 2064)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_products_in_a_row(M, C, K, dtype):
    """Calls that nothing waits between, few and many channels to many and few tokens."""
    a, w = ints(M, K, 40).cuda(), ints(C, K, 41).cuda()
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    sa, sw, ws = one(M), one(C), sv.new_matmul_workspace(M, C, K)
    want = (a.double() @ w.double().t()).float().to(dtype)
    outs = [sv.int8_matmul(a, sa, w, sw, dtype=dtype, workspace=ws)["out"] for _ in range(30)]
    torch.cuda.synchronize()
    assert sv.read_status(ws) == 0 and all(torch.equal(o, want) for o in outs)


def test_empty_calls():
    e = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    assert sv.residual_norm(e(0, 64), e(0, 64), quantize=True)["out"].shape == (0, 64)
    assert sv.quantize_rows(e(2, 0, 64))["scale"].shape == (2, 0)
    i8 = torch.int8
    assert sv.int8_matmul(e(0, 64, dtype=i8), e(0, dtype=F32), e(5, 64, dtype=i8), e(5, dtype=F32))["out"].shape == (0, 5)
    assert sv.process_logits(e(0, 3, 100))["out"].shape == (0, 3, 100)
    assert sv.process_logits(e(3, 0, 100))["out"].shape == (3, 0, 100)


def test_no_gradients_are_recorded():
    x = torch.randn(2, 64, device="cuda", requires_grad=True)
    assert not sv.residual_norm(x)["out"].requires_grad and not sv.process_logits(x[None])["out"].requires_grad
