"""Calls on another stream than the current one: what they allocate themselves is theirs until that stream has passed
them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SLEEP = 20_000_000              # GPU cycles, some ten milliseconds


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


class Layer:
    """Inputs of a layer over NF4, two of them stacked, and over bf16, and the calls with scratch of their own."""

    def __init__(self, M, K=1024, N=2048, r=16):
        q, g = qlib(), torch.Generator(device=DEV)
        g.manual_seed(M)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=DEV) * std).to(BF)

        self.X, self.dY, self.W = normal(M, K), normal(M, N), normal(N, K, std=0.05)
        self.L1, self.L2 = normal(K, r, std=K ** -0.5), normal(r, N, std=0.1)
        self.G1, self.G2 = normal(2, K, r, std=K ** -0.5), normal(2, r, N // 2, std=0.1)
        codes, absmax = q.nf4_quantize(self.W)
        self.base = (codes, *q.nf4_double_quant(absmax))
        self.N = N

    def calls(self, q, **kw):
        X, dY, base, N, L1, L2 = self.X, self.dY, self.base, self.N, self.L1, self.L2
        yield "qlora_linear_fwd", q.qlora_linear_fwd(X, *base, N, L1, L2, 1.5, **kw)
        yield "qlora_linear_bwd", q.qlora_linear_bwd(X, dY, *base, L1, L2, 1.5, **kw)
        if X.shape[0] > 16:
            yield "qlora_group_fwd", q.qlora_group_fwd(X, *base, N // 2, 2, self.G1, self.G2, 1.5, **kw)
            yield "qlora_group_bwd", q.qlora_group_bwd(X, dY, *base, 2, self.G1, self.G2, 1.5, **kw)
        yield "qlora_lora_down", q.qlora_lora_down(X, L1, **kw)
        yield "qlora_lora_grad_in", q.qlora_lora_grad_in(dY, L2, 1.5, **kw)
        yield "lora_linear_fwd", q.lora_linear_fwd(X, self.W, L1, L2, 1.5, **kw)
        yield "lora_linear_bwd", q.lora_linear_bwd(X, dY, self.W, L1, L2, 1.5, **kw)
        yield "qlora_linear_fwd_dropout", q.qlora_linear_fwd_dropout(X, *base, N, L1, L2, 1.5, p=0.1, seed=1, **kw)
        yield "qlora_linear_bwd_dropout", q.qlora_linear_bwd_dropout(X, dY, *base, L1, L2, 1.5, p=0.1, seed=1, **kw)


def tensors(v):
    return [t for t in (v if isinstance(v, tuple) else (v,)) if t is not None]


@pytest.mark.parametrize("M", [8, 512])
def test_scratch_outlives_a_call_on_another_stream(M, monkeypatch):
    """Memory that the current stream takes right after the call, which still waits, is not the call's scratch."""
    from bit_quantized_lora_blockwise_amd import _lib
    q, d = qlib(), Layer(M)
    side, scratch, own = torch.cuda.Stream(), [], _lib._workspace

    def seen(*args):
        ws = own(*args)
        scratch.append((ws.data_ptr(), ws.numel()))
        return ws

    plain = dict(d.calls(q))
    monkeypatch.setattr(_lib, "_workspace", seen)
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)                     # the calls wait behind this
    for name, got in d.calls(q, stream=side):
        at, n = scratch[-1]
        taken = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
        assert at not in [t.data_ptr() for t in taken], name
        plain[name] = (plain[name], got)
    torch.cuda.synchronize()
    assert len(scratch) == len(plain)
    for name, (want, got) in plain.items():
        for a, b in zip(tensors(want), tensors(got)):
            assert torch.equal(a, b), name


def test_scratch_is_not_what_the_current_stream_may_still_use():
    """A block that a call on the current stream has just let go of, with its work still queued."""
    from bit_quantized_lora_blockwise_amd import _lib
    like, side = torch.empty(1, device=DEV), torch.cuda.Stream()
    for n in (1000, 3 << 20):
        first = _lib._workspace(n, like, None, None)
        held = first.data_ptr()
        del first
        other = _lib._workspace(n, like, None, side).data_ptr()
        again = _lib._workspace(n, like, None, torch.cuda.current_stream()).data_ptr()
        assert other != held and again == held


def test_outputs_outlive_a_call_on_another_stream():
    """An output that the call allocates: let go of while the call still waits, it is not handed to the current stream;
    nor is what that stream has just let go of, with its work queued, taken for one."""
    q, d = qlib(), Layer(40)
    codes, c2, c1 = d.base
    absmax = q.nf4_quantize(d.W)[1]
    q4c, q4a = q.q4_quantize(d.W, "fp4")
    w, wt = q.mx4_quantize(d.W), q.mx4_quantize(d.W, transpose=True)
    x = q.mx4_quantize(d.X)
    T, G = q.qlora_lora_down(d.X, d.L1), q.qlora_lora_grad_in(d.dY, d.L2)
    N, K = d.W.shape
    calls = {
        "nf4_quantize": lambda **k: q.nf4_quantize(d.W, **k),
        "nf4_quantize_dq": lambda **k: q.nf4_quantize_dq(d.W, absmax=True, **k),
        "nf4_double_quant": lambda **k: q.nf4_double_quant(absmax, **k),
        "nf4_dequantize": lambda **k: q.nf4_dequantize(*d.base, N, K, **k),
        "q4_quantize": lambda **k: q.q4_quantize(d.W, "fp4", **k),
        "q4_double_quant": lambda **k: q.q4_double_quant(q4a, "mean", **k),
        "q4_dequantize": lambda **k: q.q4_dequantize(q4c, N, K, "fp4", "absmax", absmax=q4a, **k),
        "qlora_merge": lambda **k: q.qlora_merge(*d.base, N, K, d.L1, d.L2, **k),
        "qlora_linear_fwd_t": lambda **k: q.qlora_linear_fwd_t(d.X, *d.base, N, T, d.L2, **k),
        "qlora_linear_dx": lambda **k: q.qlora_linear_dx(d.dY, *d.base, K, G, d.L1, **k),
        "lora_linear_fwd_t": lambda **k: q.lora_linear_fwd_t(d.X, d.W, T, d.L2, **k),
        "lora_linear_dx": lambda **k: q.lora_linear_dx(d.dY, d.W, G, d.L1, **k),
        "lora_dropout": lambda **k: q.lora_dropout(d.X, 0.1, 1, **k),
        "mx4_quantize": lambda **k: q.mx4_quantize(d.X, **k),
        "mx4_dequantize": lambda **k: q.mx4_dequantize(*w, N, K, **k),
        "mx4_matmul": lambda **k: q.mx4_matmul(*x, 40, *w, N, K, **k),
        "mx4_linear_fwd": lambda **k: q.mx4_linear_fwd(d.X, *w, N, d.L1, d.L2, T_out=True, p=0.1, **k),
        "mx4_linear_bwd": lambda **k: q.mx4_linear_bwd(d.X, d.dY, *wt, d.L1, d.L2, T=T, **k),
    }
    for name, _ in d.calls(q):
        calls[name] = lambda name=name, **k: dict(d.calls(q, **k))[name]
    side = torch.cuda.Stream()
    for name, call in calls.items():
        own = tensors(call())
        sizes = [t.numel() * t.element_size() for t in own]
        held = {t.data_ptr() for t in own}
        keep = [t.clone() for t in own]
        del own
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLEEP)
        got = tensors(call(stream=side))
        at = {t.data_ptr() for t in got}
        assert not at & held, name
        side.synchronize()
        for a, b in zip(keep, got):
            assert torch.equal(a, b), name
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLEEP)
        at = {t.data_ptr() for t in tensors(call(stream=side))}      # and gone at once
        taken = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
        assert not at & {t.data_ptr() for t in taken}, name
        torch.cuda.synchronize()
        del got, taken


def test_stream_by_its_handle_alone():
    """An object that holds a stream's handle, from another library say, does for a stream."""
    class Handle:
        cuda_stream = torch.cuda.Stream().cuda_stream

    q, d = qlib(), Layer(40)
    plain = dict(d.calls(q))
    torch.cuda.synchronize()
    for name, got in d.calls(q, stream=Handle):
        torch.cuda.synchronize()
        for a, b in zip(tensors(plain[name]), tensors(got)):
            assert torch.equal(a, b), name
