"""The decode operators on operands past 4 GiB: rows and experts behind that offset give
what they give in an operand of their own."""

import numpy as np
import pytest

from tests import decode_cases as dc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield
    torch.cuda.empty_cache()


def test_linear_weights_and_rows():
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(1)
    N, K, some = 300000, 32768, 40
    codes, scales = dc.weights(rng, "mxfp4", (some,), K)
    c = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(N, K // 32, dtype=torch.uint8, device="cuda")
    at = torch.cat([torch.arange(some // 2), torch.arange(N - some // 2, N)]).cuda()
    c[at], s[at] = dc.dev(codes), dc.dev(scales)
    # Rows of activations 2^30 elements (2 GiB) apart, and the same close together.
    ld = 1 << 30
    far = torch.zeros(2 * ld + K, dtype=torch.bfloat16, device="cuda").as_strided((3, K), (ld, 1))
    x = dc.dev_bf16(dc.bf16(rng.standard_normal((3, K)))[1])
    far.copy_(x)
    for M in (1, 3):
        got = wush.linear_w4("mxfp4", far[:M], c, s, out_dtype=torch.float32)
        # The same shape of workgroup, so the same order of sums.
        cut, cut_s = c[-16384:].clone(), s[-16384:].clone()
        cut[: some // 2], cut_s[: some // 2] = c[: some // 2], s[: some // 2]
        want = wush.linear_w4("mxfp4", x[:M], cut, cut_s, out_dtype=torch.float32)
        assert torch.equal(got[:, : some // 2], want[:, : some // 2])
        assert torch.equal(got[:, -some // 2 :], want[:, -some // 2 :])
        assert float(got[:, -some // 2 :].abs().min()) > 0
        assert torch.all(got[:, some // 2 : -some // 2] == 0)


def test_experts():
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(2)
    E, H, I = 160, 8192, 4096
    gc, gs = dc.weights(rng, "mxfp4", (2 * I,), H)
    wc, ws = dc.weights(rng, "mxfp4", (H,), I)
    last = 4

    def spread(codes, scales, n):
        c = torch.zeros(n, *codes.shape, dtype=torch.uint8, device="cuda")
        s = torch.zeros(n, *scales.shape, dtype=torch.uint8, device="cuda")
        c[-1], s[-1] = dc.dev(codes), dc.dev(scales)
        return wush.W4Experts(c, s)

    x = dc.dev_bf16(dc.bf16(rng.standard_normal((2, H)))[1])
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    router[E - 1] = x[0] / 1024  # the first token's first choice
    gate_up, down = spread(gc, gs, E), spread(wc, ws, E)
    got = wush.moe_w4("mxfp4", x, router, gate_up, down, 2, out_dtype=torch.float32)
    small = wush.moe_w4("mxfp4", x, router[-last:].contiguous(), wush.W4Experts(*(t[-last:].contiguous() for t in gate_up[:2])),
                        wush.W4Experts(*(t[-last:].contiguous() for t in down[:2])), 2, out_dtype=torch.float32)
    assert int(got.ids[0, 0]) == E - 1 and int(small.ids[0, 0]) == last - 1
    assert torch.equal(got.weights[0], small.weights[0])
    assert torch.equal(got.out[0], small.out[0]) and float(got.out[0].abs().max()) > 0


def test_logits():
    import mxfp4_activation_amd as wush

    R, V = 70000, 32800
    logits = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    ends = torch.randn(2, 64, V, generator=gen, device="cuda").to(torch.bfloat16)
    logits[:64], logits[-64:] = ends[0], ends[1]
    t = torch.randint(0, V, (R,), generator=gen, device="cuda")
    got = wush.token_logprobs(logits, t, top=3)
    for part, at in ((ends[0], slice(0, 64)), (ends[1], slice(R - 64, R))):
        want = wush.token_logprobs(part.contiguous(), t[at].contiguous(), top=3)
        assert torch.equal(got.top_ids[at], want.top_ids)
        for a, b in zip(got, want):
            assert torch.allclose(a[at].float(), b.float(), rtol=2.0**-20, atol=2.0**-18)
    middle = float(np.log(V))
    assert torch.allclose(got.entropy[64:-64], torch.full_like(got.entropy[64:-64], middle), rtol=2.0**-20)
    assert torch.all(got.top_ids[64:-64] == torch.arange(3, device="cuda", dtype=torch.int32))
