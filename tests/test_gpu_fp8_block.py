"""GPU parity of the block-scaled FP8 quantizers and product against plain
references (block_ref.py).

Codes and scales are taken in the same fp32 arithmetic on both sides and must
match bit for bit.  The product must stay within block_ref's bound, which
follows from how the fp8 matrix instructions add.
"""
import numpy as np
import pytest

import block_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int8_quantized_matmul_row_amd as pkg
    pkg.lib()  # fails loudly when the library is missing


def torch_dtype(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def values(codes):
    import torch
    return codes.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)


def rand(shape, seed, dtype, scale=1.0, outliers=True):
    """16-bit normals with a few large columns, a zero block and signed zeros."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn(*shape, generator=g)
    if outliers:
        x[..., :: max(1, shape[-1] // 3)] *= 30.0
        x[..., 5] = -0.0
    return x.to(torch_dtype(dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 64), (1, 128), (2, 192), (15, 256), (16, 640), (17, 1024), (100, 4160),
                                 (333, 576)])
def test_act_codes(M, K, dtype):
    import torch
    import int8_quantized_matmul_row_amd as pkg
    x = rand((M, K), M + K, dtype)
    x[0, :64] = 0                                    # a block of zeros, or half of one
    if M > 1:
        x[M - 1] = torch.finfo(x.dtype).tiny / 4     # subnormal values
        x[M // 2, K - 1] = torch.finfo(torch.float16).max
    q = pkg.quantize_act_fp8_block(x.cuda())
    codes, scales = ref.quantize(x.float().numpy(), 1)
    assert tuple(q.SCA.shape) == (ref.blocks(K), M)
    assert np.array_equal(q.SCA.cpu().numpy().T, scales)
    assert np.array_equal(values(q.CA), codes)
    assert np.array_equal(np.signbit(values(q.CA)), np.signbit(codes))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 64), (127, 128), (128, 192), (129, 256), (300, 1024), (3, 100, 320),
                                   (2, 2, 130, 192)])
def test_weight_codes(shape, dtype):
    import int8_quantized_matmul_row_amd as pkg
    w = rand(shape, sum(shape), dtype, 0.02)
    w[..., 0, :] = 0
    CB, SCB = pkg.quantize_weight_fp8_block(w.cuda())
    N, K = shape[-2:]
    flat = w.float().numpy().reshape(-1, N, K)
    cb, scb = values(CB).reshape(-1, N, K), SCB.cpu().numpy().reshape(-1, ref.blocks(N), ref.blocks(K))
    for i in range(flat.shape[0]):
        codes, scales = ref.quantize(flat[i], 128)
        assert np.array_equal(scb[i], scales)
        assert np.array_equal(cb[i], codes)


def random_codes(shape, seed):
    """Codes of every finite E4M3 value."""
    import torch
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 127, shape, generator=g, dtype=torch.uint8)
    return c | (torch.randint(0, 2, shape, generator=g, dtype=torch.uint8) << 7)


SHAPES = [(1, 1, 64), (1, 130, 128), (2, 16, 192), (3, 500, 1024), (7, 129, 640), (8, 64, 2048), (15, 33, 256),
          (16, 256, 448), (17, 257, 576), (31, 128, 1088), (32, 300, 4160), (33, 100, 320), (63, 260, 512),
          (64, 513, 128), (65, 31, 704), (100, 200, 192), (129, 255, 256), (200, 384, 640), (333, 77, 832),
          (513, 257, 320), (600, 520, 192), (1030, 96, 128)]


@pytest.mark.parametrize("dtype,bias", [("f16", True), ("bf16", False)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, dtype, bias):
    import torch
    import int8_quantized_matmul_row_amd as pkg
    g = torch.Generator().manual_seed(7 * M + N + K)
    CA, CB = random_codes((M, K), M + 1), random_codes((N, K), N + 2)
    # scales spread over four octaves, each block its own: a wrong scale shows
    SCA = torch.exp2(4 * torch.rand(ref.blocks(K), M, generator=g) - 2)
    SCB = 0.02 * torch.exp2(4 * torch.rand(ref.blocks(N), ref.blocks(K), generator=g) - 2)
    b = (torch.randn(N, generator=g)).to(torch_dtype(dtype)) if bias else None
    q = pkg.BlockAct(CA.cuda(), SCA.cuda(), pkg.F16 if dtype == "f16" else pkg.BF16)
    Y = pkg.matmul_fp8_block(q, CB.cuda(), SCB.cuda(), bias=None if b is None else b.cuda())
    assert Y.dtype == torch_dtype(dtype) and tuple(Y.shape) == (M, N)
    want, bound = ref.product(values(CA), SCA.numpy().T, values(CB), SCB.numpy(),
                              None if b is None else b.float().numpy().astype(np.float64))
    err = np.abs(Y.float().cpu().numpy().astype(np.float64) - want)
    worst = (err / (bound + 2 * ref.half_step16(np.abs(want) + bound, dtype == "bf16"))).max()
    print(f"{M}x{N}x{K} {dtype}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0


# (large tiles, tall tiles, K split over workgroups, a ragged edge of each)
LARGE = [(2048, 4096, 320), (1000, 4096, 192), (512, 28672, 192), (257, 28700, 448), (64, 16384, 640),
         (40, 600, 8192), (200, 300, 4160), (63, 4095, 4096), (4100, 1000, 192), (3000, 2050, 128), (129, 129, 2048),
         (450, 8192, 576), (17, 100, 1344)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_product_at_sampled_outputs(M, N, K, dtype):
    import torch
    import int8_quantized_matmul_row_amd as pkg
    g = torch.Generator().manual_seed(M + N + K)
    CA, CB = random_codes((M, K), M + 1).cuda(), random_codes((N, K), N + 2).cuda()
    SCA = torch.exp2(4 * torch.rand(ref.blocks(K), M, generator=g) - 2)
    SCB = 0.02 * torch.exp2(4 * torch.rand(ref.blocks(N), ref.blocks(K), generator=g) - 2)
    b = torch.randn(N, generator=g).to(torch_dtype(dtype))
    q = pkg.BlockAct(CA, SCA.cuda(), pkg.F16 if dtype == "f16" else pkg.BF16)
    Y = pkg.matmul_fp8_block(q, CB, SCB.cuda(), bias=b.cuda())
    rows = np.unique(np.r_[0, M - 1, np.random.default_rng(M).integers(0, M, 40)])
    cols = np.unique(np.r_[0, N - 1, np.random.default_rng(N).integers(0, N, 60)])
    A = values(CA[rows]) * ref.spread(SCA.numpy().T[rows], 1, len(rows), K)
    W = values(CB[cols]) * ref.spread(SCB.numpy()[cols // 128], 1, len(cols), K)
    want = A @ W.T + b.float().numpy().astype(np.float64)[cols]
    bound = ref.product_bound(A, W, want)
    err = np.abs(Y.float().cpu().numpy().astype(np.float64)[np.ix_(rows, cols)] - want)
    worst = (err / (bound + 2 * ref.half_step16(np.abs(want) + bound, dtype == "bf16"))).max()
    print(f"{M}x{N}x{K} {dtype}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0
    # the same bits again (split K adds its parts in order)
    again = pkg.matmul_fp8_block(q, CB, SCB.cuda(), bias=b.cuda())
    assert torch.equal(Y, again)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (1, 200, 4160), (4, 128, 8192), (8, 96, 1024), (9, 300, 448), (16, 512, 192), (20, 130, 640),
                                   (64, 200, 320), (70, 256, 1024), (300, 130, 192), (700, 300, 256),
                                   (40, 130, 4160)])
def test_linear(M, N, K, dtype):
    """The one-call forward: codes as the quantizer gives them, then the product."""
    import int8_quantized_matmul_row_amd as pkg
    x, w = rand((M, K), M, dtype), rand((N, K), N, dtype, 0.02)
    CB, SCB = pkg.quantize_weight_fp8_block(w.cuda())
    bias = rand((N,), K, dtype, 0.5, outliers=False)
    Y = pkg.linear_fp8_block(x.cuda(), CB, SCB, bias=bias.cuda())
    ca, sa = ref.quantize(x.float().numpy(), 1)
    want, bound = ref.product(ca, sa, values(CB), SCB.cpu().numpy(), bias.float().numpy().astype(np.float64))
    err = np.abs(Y.float().cpu().numpy().astype(np.float64) - want)
    worst = (err / (bound + 2 * ref.half_step16(np.abs(want) + bound, dtype == "bf16"))).max()
    print(f"linear {M}x{N}x{K} {dtype}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0
    # a second call on the same buffers gives the same bits
    again = pkg.linear_fp8_block(x.cuda(), CB, SCB, bias=bias.cuda(), out=Y.clone())
    assert (again == Y).all()


@pytest.mark.parametrize("M,N", [(0, 128), (5, 0), (0, 0)])
def test_empty(M, N):
    import torch
    import int8_quantized_matmul_row_amd as pkg
    x = torch.zeros(M, 128, dtype=torch.float16, device="cuda")
    CB, SCB = pkg.quantize_weight_fp8_block(torch.zeros(N, 128, dtype=torch.float16, device="cuda"))
    assert tuple(SCB.shape) == (ref.blocks(N), 1)
    assert tuple(pkg.linear_fp8_block(x, CB, SCB).shape) == (M, N)
    q = pkg.quantize_act_fp8_block(x)
    assert tuple(pkg.matmul_fp8_block(q, CB, SCB).shape) == (M, N)


@pytest.mark.parametrize("M", [4, 300])
def test_another_stream(M):
    """Work given to a stream that is not the current one waits for it and is
    whole when it is done."""
    import torch
    import int8_quantized_matmul_row_amd as pkg
    x, w = rand((M, 1024), 3, "bf16").cuda(), rand((500, 1024), 4, "bf16", 0.02).cuda()
    CB, SCB = pkg.quantize_weight_fp8_block(w)
    want = pkg.linear_fp8_block(x, CB, SCB)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [pkg.linear_fp8_block(x, CB, SCB, stream=s) for _ in range(5)]
    s.synchronize()
    assert all(torch.equal(y, want) for y in got)


@pytest.mark.parametrize("M", [2, 80])
def test_weight_past_two_gib(M):
    """Rows of a weight whose codes pass 2^31 and 2^32 bytes."""
    import torch
    import int8_quantized_matmul_row_amd as pkg
    K, N = 16384, 270000
    assert N * K > 1 << 32
    CB = random_codes((1000, K), 5).cuda().repeat(270, 1)
    SCB = torch.ones(ref.blocks(N), ref.blocks(K), device="cuda")
    SCB[-1] = 3.0
    x = rand((M, K), 6, "f16", outliers=False).cuda()
    Y = pkg.linear_fp8_block(x, CB, 0.02 * SCB)
    ca, sa = ref.quantize(x.float().cpu().numpy(), 1)
    for n in (0, 131072 - 40, 262144 - 40, N - N % 128 - 40):  # 2^31, 2^32 bytes, the last block's first row
        rows = slice(n, n + 80)
        scale = np.ones((80, 1))
        scale[np.arange(n, n + 80) >= N - N % 128] = 3.0
        codes = values(CB[rows]) * scale
        want, bound = ref.product(ca[:4], sa[:4], codes, np.full((1, ref.blocks(K)), 0.02, np.float32))
        err = np.abs(Y[:4, rows].float().cpu().numpy().astype(np.float64) - want)
        assert (err <= bound + 2 * ref.half_step16(np.abs(want) + bound, False)).all()
    # every repetition of the 1000 rows gives the same outputs, up to the last block
    same = Y[:, : 269 * 1000].view(M, 269, 1000)
    assert torch.equal(same, same[:, :1].expand_as(same))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 192), (3, 300, 576), (33, 130, 4160), (300, 300, 320), (1200, 1000, 192)])
def test_a_value_that_is_not_finite_shows_in_its_row_alone(M, N, K, value, dtype):
    """One NaN or infinity in a row of X: a code that is NaN, hence NaN in all of the
    row's outputs, whichever kernel runs; the other rows' are untouched."""
    import torch
    import int8_quantized_matmul_row_amd as pkg
    x = rand((M, K), 1, dtype).cuda()
    q = pkg.quantize_weight_fp8_block(rand((N, K), 2, dtype).cuda())
    was = pkg.linear_fp8_block(x, *q)
    x[M // 2, K - 3] = float(value)
    Y = pkg.linear_fp8_block(x, *q)
    assert Y[M // 2].isnan().all()
    others = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(Y[others], was[others]) and torch.isfinite(was).all()
