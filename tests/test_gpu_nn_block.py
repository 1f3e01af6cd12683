"""LinearFP8Block and MoEFFN8bit on the GPU: quantized once when placed, forward
against the binding's own steps and, end to end, against 64 bits."""
import numpy as np
import pytest

import block_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("lead", [(1,), (2, 9), (3, 0)])
def test_linear_layer(lead, dtype):
    import torch
    import int8_quantized_matmul_row_amd as pkg
    from int8_quantized_matmul_row_amd import nn as n8
    dt = getattr(torch, dtype)
    lin = torch.nn.Linear(192, 100, dtype=dt)
    m = n8.LinearFP8Block.from_linear(lin)
    assert not m.quantized and m.weight is not None
    with pytest.raises(RuntimeError, match="GPU only"):
        m(torch.zeros(1, 192, dtype=dt))
    m = m.cuda()
    assert m.quantized and m.weight is None and m.CB.dtype == torch.uint8
    codes = m.CB.clone()
    m = m.to(dt).cuda()
    assert torch.equal(m.CB, codes) and m.SCB.dtype == torch.float32
    x = torch.randn(*lead, 192, dtype=dt, device="cuda")
    y = m(x)
    assert y.shape == (*lead, 100) and y.dtype == dt
    CB, SCB = pkg.quantize_weight_fp8_block(lin.weight.data.cuda())
    assert torch.equal(CB, m.CB) and torch.equal(SCB, m.SCB)
    want = pkg.linear_fp8_block(x.reshape(-1, 192), CB, SCB, bias=lin.bias.data.cuda())
    assert torch.equal(y.reshape(-1, 100), want)


@pytest.mark.parametrize("kw", [dict(top_k=2), dict(top_k=3, scoring="sigmoid", n_group=4, topk_group=2, scale=2.5)])
@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_mixture(tokens, kw):
    """Router, routing and experts as a model runs them, with padding, a strided
    input, and a copy moved off the GPU and back."""
    import torch
    import int8_quantized_matmul_row_amd as pkg
    from int8_quantized_matmul_row_amd import nn as n8
    E, K, I = 16, 256, 192
    g = torch.Generator().manual_seed(tokens)
    bf = torch.bfloat16
    router = (torch.randn(E, K, generator=g) / 16).to(bf)
    gate, up = ((torch.randn(E, I, K, generator=g) / 16).to(bf) for _ in range(2))
    down = (torch.randn(E, K, I, generator=g) / 14).to(bf)
    bias = 0.1 * torch.randn(E, generator=g) if "scoring" in kw else None
    m = n8.MoEFFN8bit(router, gate, up, down, balance_bias=bias, **kw).cuda()
    assert m.quantized and m.W13 is None
    m = m.cpu().cuda()
    wide = torch.randn(1, tokens, 2 * K, generator=g).to(bf).cuda()
    x = wide[..., ::2]
    keep = torch.ones(1, tokens, dtype=torch.bool, device="cuda")
    keep[0, tokens // 2] = tokens == 1
    y = m(x, keep=keep)
    assert y.shape == x.shape
    ids = m.last_ids.cpu().numpy()
    if tokens > 1:
        assert (ids[tokens // 2] == -1).all() and (y[0, tokens // 2] == 0).all()
    X = x.reshape(-1, K).contiguous()
    logits = torch.nn.functional.linear(X, router.cuda()).masked_fill(~keep.reshape(-1, 1), float("-inf"))
    route = {k: v for k, v in kw.items() if k != "top_k"}
    i2, w2 = pkg.route_experts(logits, kw["top_k"], bias=None if bias is None else bias.cuda(), **route)
    assert (i2.cpu().numpy() == ids).all()

    def values(CB, SCB):
        c = CB.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
        flat, s = c.reshape(-1, *c.shape[-2:]), SCB.cpu().numpy().reshape(-1, *SCB.shape[-2:])
        return np.stack([f * ref.spread(t, 128, *f.shape) for f, t in zip(flat, s)]).reshape(c.shape)

    codes, scales = ref.quantize(X.float().cpu().numpy(), 1)
    want, bound = ref.experts(codes * ref.spread(scales, 1, tokens, K), ids, w2.cpu().numpy(),
                              values(m.CB13, m.SCB13), values(m.CB2, m.SCB2))
    err = np.abs(y.reshape(-1, K).float().cpu().numpy().astype(np.float64) - want)
    assert (err <= bound + 2 * ref.half_step16(np.abs(want) + bound, True)).all()


def test_refusals():
    import torch
    from int8_quantized_matmul_row_amd import nn as n8
    h = torch.float16
    with pytest.raises(ValueError, match="multiple of 64"):
        n8.LinearFP8Block(torch.zeros(8, 100, dtype=h))
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        n8.LinearFP8Block(torch.zeros(8, 128))
    args = [torch.zeros(4, 128, dtype=h), torch.zeros(4, 64, 128, dtype=h), torch.zeros(4, 64, 128, dtype=h),
            torch.zeros(4, 128, 64, dtype=h)]
    with pytest.raises(ValueError, match="belong together"):
        n8.MoEFFN8bit(*args[:3], torch.zeros(4, 64, 128, dtype=h), top_k=2)
    m = n8.MoEFFN8bit(*args, top_k=2)
    with pytest.raises(RuntimeError, match="GPU only"):
        m(torch.zeros(1, 128, dtype=h))
    with pytest.raises(ValueError, match="features"):
        m.cuda()(torch.zeros(1, 64, dtype=h, device="cuda"))
