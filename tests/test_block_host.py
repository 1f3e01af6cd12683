"""The block-scaled FP8, routing and expert entry points on the CPU: bad
arguments are refused before any HIP call (fake addresses, never dereferenced),
and the torch-level binding refuses tensors of the wrong type, shape or place
before any pointer reaches the library."""
import ctypes

import pytest

import int8_quantized_matmul_row_amd as pkg
from test_binding_host import FakeStream, FakeTensor, FakeTorch, FakeLib

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 0x10000


def qw(W=A, dtype=0, batch=1, N=8, K=64, CB=A, SCB=A):
    return pkg.lib().llmint8_quantize_weight_fp8_block(W, dtype, batch, N, K, CB, SCB, None)


def qa(X=A, dtype=0, M=8, K=64, CA=A, SCA=A):
    return pkg.lib().llmint8_quantize_act_fp8_block(X, dtype, M, K, CA, SCA, None)


def mm(dtype=0, M=8, N=8, K=64, CA=A, SCA=A, CB=A, SCB=A, bias=None, Y=A, ws=A, wsb=1 << 40):
    return pkg.lib().llmint8_matmul_fp8_block(dtype, M, N, K, CA, SCA, CB, SCB, bias, Y, ws, wsb, None)


def lin(X=A, dtype=0, M=8, N=8, K=64, CB=A, SCB=A, bias=None, Y=A, ws=A, wsb=1 << 40):
    return pkg.lib().llmint8_linear_fp8_block(X, dtype, M, N, K, CB, SCB, bias, Y, ws, wsb, None)


def route(logits=A, dtype=2, T=4, E=64, bias=None, scoring=0, n_group=1, topk_group=1, k=4, renorm=1, ids=A, w=A):
    return pkg.lib().llmint8_route_experts(logits, dtype, T, E, bias, scoring, n_group, topk_group, k, renorm,
                                           ctypes.c_float(1.0), ids, w, None)


def experts(X=A, dtype=0, T=4, K=128, I=64, E=8, k=2, ids=A, w=A, CB13=A, SCB13=A, CB2=A, SCB2=A, Y=A, ws=A,
            wsb=1 << 40):
    return pkg.lib().llmint8_experts_fp8_block(X, dtype, T, K, I, E, k, ids, w, CB13, SCB13, CB2, SCB2, Y, ws, wsb,
                                               None)


def test_quantizers_refuse():
    for f in (qw, qa):
        assert f(dtype=2) == INVALID
        assert f(dtype=-1) == INVALID
        assert f(K=-64) == INVALID
        assert f(K=0) == UNSUPPORTED
        assert f(K=100) == UNSUPPORTED
        assert f(K=pkg.K_MAX + 64) == UNSUPPORTED
    assert qw(N=-1) == INVALID and qw(batch=-1) == INVALID and qa(M=-1) == INVALID
    assert qw(N=(1 << 30) + 1) == UNSUPPORTED
    assert qw(batch=1 << 24, N=129) == UNSUPPORTED
    assert qa(M=1 << 31) == UNSUPPORTED
    for name in ("W", "CB", "SCB"):
        assert qw(**{name: None}) == INVALID and qw(**{name: A + 4}) == INVALID
    for name in ("X", "CA", "SCA"):
        assert qa(**{name: None}) == INVALID and qa(**{name: A + 4}) == INVALID
    assert qw(N=0, W=None, CB=None, SCB=None) == OK
    assert qw(batch=0, W=None, CB=None, SCB=None) == OK
    assert qa(M=0, X=None, CA=None, SCA=None) == OK


def test_products_refuse():
    for f in (mm, lin):
        assert f(dtype=2) == INVALID
        assert f(M=-1) == INVALID and f(N=-1) == INVALID
        assert f(K=96) == UNSUPPORTED and f(N=(1 << 30) + 1) == UNSUPPORTED and f(M=1 << 31) == UNSUPPORTED
        for name in ("CB", "SCB", "Y"):
            assert f(**{name: None}) == INVALID and f(**{name: A + 2}) == INVALID
        assert f(bias=A + 2) == INVALID
        assert f(ws=A + 4) == INVALID
        assert f(M=0, CB=None, Y=None, ws=None, wsb=0) == OK and f(N=0, CB=None, Y=None, ws=None, wsb=0) == OK
    assert mm(CA=None) == INVALID and mm(SCA=A + 4) == INVALID and lin(X=None) == INVALID
    for M, N, K in ((1, 4096, 4096), (100, 300, 192), (2048, 16384, 4096)):
        need = pkg.llmint8_linear_fp8_block_workspace_size(M, N, K)
        if need:
            assert lin(M=M, N=N, K=K, ws=None) == INVALID
            assert lin(M=M, N=N, K=K, wsb=need - 1) == INVALID
        need = pkg.llmint8_matmul_fp8_block_workspace_size(M, N, K)
        if need:
            assert mm(M=M, N=N, K=K, ws=None) == INVALID
            assert mm(M=M, N=N, K=K, wsb=need - 1) == INVALID


def test_route_refuses():
    assert route(dtype=3) == INVALID and route(dtype=-1) == INVALID
    assert route(scoring=2) == INVALID and route(scoring=-1) == INVALID
    assert route(T=-1) == INVALID and route(E=0) == INVALID
    assert route(n_group=0) == INVALID and route(n_group=7) == INVALID
    assert route(n_group=8, topk_group=0) == INVALID and route(n_group=8, topk_group=9) == INVALID
    assert route(k=0) == INVALID and route(k=65) == INVALID
    assert route(n_group=8, topk_group=2, k=17) == INVALID   # 16 experts in two groups
    assert route(E=1025) == UNSUPPORTED and route(k=33) == UNSUPPORTED and route(T=1 << 31) == UNSUPPORTED
    assert route(E=650, n_group=65, topk_group=4) == UNSUPPORTED
    for name in ("logits", "ids", "w"):
        assert route(**{name: None}) == INVALID and route(**{name: A + 4}) == INVALID
    assert route(bias=A + 4) == INVALID
    assert route(T=0, logits=None, ids=None, w=None) == OK


def test_experts_refuse():
    assert experts(dtype=2) == INVALID
    assert experts(T=-1) == INVALID and experts(E=0) == INVALID and experts(k=0) == INVALID
    assert experts(K=100) == UNSUPPORTED and experts(I=32) == UNSUPPORTED and experts(I=0) == UNSUPPORTED
    assert experts(E=1025) == UNSUPPORTED and experts(k=33) == UNSUPPORTED and experts(T=1 << 31) == UNSUPPORTED
    assert experts(K=65536, I=32768) == UNSUPPORTED   # 2 I K reaches 2^32
    for name in ("X", "ids", "w", "CB13", "SCB13", "CB2", "SCB2", "Y", "ws"):
        assert experts(**{name: None}) == INVALID and experts(**{name: A + 4}) == INVALID
    need = pkg.llmint8_experts_fp8_block_workspace_size(4, 8, 2, 128, 64)
    assert need > 0 and experts(wsb=need - 1) == INVALID
    assert experts(T=0, X=None, ids=None, w=None, CB13=None, Y=None, ws=None, wsb=0) == OK


def test_workspace_sizes_of_bad_shapes_are_zero():
    for M, N, K in ((-1, 8, 64), (8, 8, 100), (8, (1 << 30) + 1, 64), (0, 8, 64), (8, 0, 64)):
        assert pkg.llmint8_matmul_fp8_block_workspace_size(M, N, K) == 0
        assert pkg.llmint8_linear_fp8_block_workspace_size(M, N, K) == 0
    for T, E, k, K, I in ((-1, 8, 2, 128, 64), (4, 0, 2, 128, 64), (4, 8, 0, 128, 64), (4, 8, 2, 100, 64),
                          (0, 8, 2, 128, 64), (4, 1025, 2, 128, 64)):
        assert pkg.llmint8_experts_fp8_block_workspace_size(T, E, k, K, I) == 0
    # the workspace of many tokens is bounded: they run in chunks
    most = pkg.llmint8_experts_fp8_block_workspace_size((1 << 31) - 1, 8, 8, 4096, 1024)
    assert 0 < most < 3 << 30


# ---- the torch-level binding -----------------------------------------------------

class Shaped(FakeTensor):
    def dim(self):
        return len(self.shape)


@pytest.fixture
def fakes(monkeypatch):
    torch, lib = FakeTorch(), FakeLib()
    torch.empty = lambda shape, dtype=None, device=None: (
        torch.allocated.append(Shaped(shape, dtype, str(device))) or torch.allocated[-1])
    monkeypatch.setattr(pkg, "_torch", lambda: torch)
    monkeypatch.setattr(pkg, "_lib", lib)
    return torch, lib


def linear_operands(M=64, N=200, K=320, **kw):
    t = dict(X=Shaped((M, K), "float16"), CB=Shaped((N, K), "uint8"), SCB=Shaped((2, 3), "float32"),
             bias=Shaped((N,), "float16"))
    t.update(kw)
    return t


@pytest.mark.parametrize("bad", [
    dict(X=Shaped((64, 320), "float32")), dict(X=Shaped((64, 320), "float16", "cpu")), dict(X=Shaped((320,), "float16")),
    dict(CB=Shaped((200, 320), "int8")), dict(CB=Shaped((200, 256), "uint8")),
    dict(CB=Shaped((200, 320), "uint8", "cuda:1")), dict(SCB=Shaped((200,), "float32")),
    dict(SCB=Shaped((2, 3), "float16")), dict(bias=Shaped((199,), "float16")), dict(bias=Shaped((200,), "bfloat16")),
    dict(out=Shaped((64, 201), "float16")), dict(out=Shaped((64, 200), "bfloat16"))])
def test_linear_refuses_tensors(fakes, bad):
    _, lib = fakes
    with pytest.raises((ValueError, TypeError)):
        pkg.linear_fp8_block(**linear_operands(**bad))
    assert not [c for c in lib.calls if not c.endswith("_workspace_size")]


def expert_operands(T=5, E=4, K=192, I=64, k=2, **kw):
    t = dict(X=Shaped((T, K), "bfloat16"), ids=Shaped((T, k), "int32"), weights=Shaped((T, k), "float32"),
             CB13=Shaped((E, 2, I, K), "uint8"), SCB13=Shaped((E, 2, 1, 2), "float32"), CB2=Shaped((E, K, I), "uint8"),
             SCB2=Shaped((E, 2, 1), "float32"))
    t.update(kw)
    return t


@pytest.mark.parametrize("bad", [
    dict(ids=Shaped((5, 2), "int64")), dict(ids=Shaped((4, 2), "int32")), dict(weights=Shaped((5, 2), "float16")),
    dict(weights=Shaped((5, 3), "float32")), dict(CB13=Shaped((4, 64, 192), "uint8")),
    dict(CB13=Shaped((4, 3, 64, 192), "uint8")), dict(SCB13=Shaped((4, 2, 2, 1), "float32")),
    dict(CB2=Shaped((4, 64, 192), "uint8")), dict(SCB2=Shaped((4, 1, 2), "float32")),
    dict(X=Shaped((5, 128), "bfloat16")), dict(X=Shaped((5, 192), "float32")), dict(out=Shaped((5, 192), "float16"))])
def test_experts_refuse_tensors(fakes, bad):
    _, lib = fakes
    with pytest.raises((ValueError, TypeError)):
        pkg.experts_fp8_block(**expert_operands(**bad))
    assert not [c for c in lib.calls if not c.endswith("_workspace_size")]


def test_route_refuses_tensors(fakes):
    _, lib = fakes
    x = Shaped((5, 64), "float32")
    for kw in (dict(scoring="relu"), dict(bias=Shaped((63,), "float32")), dict(bias=Shaped((64,), "float16")),
               dict(out=(Shaped((5, 2), "int64"), Shaped((5, 2), "float32")))):
        with pytest.raises(ValueError):
            pkg.route_experts(x, 2, **kw)
    with pytest.raises((ValueError, TypeError)):
        pkg.route_experts(Shaped((5, 64), "int32"), 2)
    with pytest.raises(ValueError):
        pkg.route_experts(Shaped((64,), "float32"), 2)
    assert lib.calls == []


def test_buffers_allocated_for_a_stream_are_recorded_on_it(fakes):
    torch, lib = fakes
    s = FakeStream(99)
    pkg.linear_fp8_block(**linear_operands(), stream=s)
    pkg.experts_fp8_block(**expert_operands(), stream=s)
    pkg.route_experts(Shaped((5, 64), "float32"), 2, stream=s)
    pkg.quantize_weight_fp8_block(Shaped((3, 130, 64), "float16"), stream=s)
    q = pkg.quantize_act_fp8_block(Shaped((7, 64), "bfloat16"), stream=s)
    assert q.dtype == pkg.BF16 and q.SCA.shape == (1, 7)
    pkg.matmul_fp8_block(q, Shaped((130, 64), "uint8"), Shaped((2, 1), "float32"), stream=s)
    ran = [c for c in lib.calls if not c.endswith("_workspace_size")]
    assert ran == ["llmint8_linear_fp8_block", "llmint8_experts_fp8_block", "llmint8_route_experts",
                   "llmint8_quantize_weight_fp8_block", "llmint8_quantize_act_fp8_block", "llmint8_matmul_fp8_block"]
    assert len(torch.allocated) == 2 + 2 + 2 + 2 + 2 + 2 and all(t.recorded == [s] for t in torch.allocated)
