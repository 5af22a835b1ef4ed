"""Memory that the binding allocates for a call belongs to the call's stream, so
that the allocator cannot hand it to another stream's work while the kernels
still use it.  On the CPU: tensors that claim to be on the device, a
library that only returns, and a record of every allocation's stream."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import fp8_block_scaled_sigmoid_amd as moe  # noqa: E402

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Device(torch.Tensor):
    """A host tensor that the binding takes for a device tensor."""
    users = None                        # streams that record_stream named

    @property
    def is_cuda(self):
        return True

    def record_stream(self, stream):
        self.users = (self.users or []) + [stream]


class Stream:
    def __init__(self):
        self.cuda_stream = id(self)


class Library:
    def __getattr__(self, name):
        return (lambda *a: 4096) if name.endswith("_bytes") else (lambda *a: 0)


_zeros = torch.zeros


def dev(*shape, dtype=BF):
    return _zeros(*shape, dtype=dtype).as_subclass(Device)


CALLS = {
    "moe_route_topk": lambda s: moe.moe_route_topk(dev(4, 128), dev(16, 128), dev(16, dtype=F32), 2,
                                                   stream=s),
    "moe_route_topk_quant_x": lambda s: moe.moe_route_topk_quant_x(
        dev(4, 128), dev(16, 128), dev(16, dtype=F32), 2, stream=s),
    "moe_route_topk_fp8": lambda s: moe.moe_route_topk_fp8(
        dev(4, 128, dtype=U8), dev(4, 1, dtype=F32), dev(128, 128, dtype=U8), dev(1, 1, dtype=F32),
        dev(128, dtype=F32), 2, stream=s),
    "moe_topk_from_scores": lambda s: moe.moe_topk_from_scores(dev(4, 16, dtype=F32),
                                                               dev(16, dtype=F32), 2, stream=s),
    "moe_permute": lambda s: moe.moe_permute(dev(4, 2, dtype=I32), 16, stream=s),
    "fp8_quant_1x128": lambda s: moe.fp8_quant_1x128(dev(4, 128), stream=s),
    "fp8_quant_128x128": lambda s: moe.fp8_quant_128x128(dev(1, 128, 128), stream=s),
    **{f"moe_grouped_gemm_fp8 {e}": lambda s, e=e: [t for t in moe.moe_grouped_gemm_fp8(
        dev(4, 128, dtype=U8), dev(4, 1, dtype=F32), dev(1, 256, 128, dtype=U8),
        dev(1, 2, 1, dtype=F32), dev(2, dtype=I32), 4, e, stream=s) if t is not None]
       for e in (moe.MOE_EPI_BF16, moe.MOE_EPI_SWIGLU_FP8, moe.MOE_EPI_F32)},
    "fp8_transpose_128x128": lambda s: moe.fp8_transpose_128x128(
        dev(1, 128, 128, dtype=U8), dev(1, 1, 1, dtype=F32), stream=s),
    "fp8_quant_tokens_128": lambda s: moe.fp8_quant_tokens_128(dev(4, 128), dev(2, dtype=I32),
                                                               stream=s),
    "moe_grouped_wgrad_fp8": lambda s: [moe.moe_grouped_wgrad_fp8(
        dev(128, 128, dtype=U8), dev(128, 1, dtype=F32), dev(128, 128, dtype=U8),
        dev(128, 1, dtype=F32), dev(2, dtype=I32), stream=s)],
    "moe_grouped_dgrad_fp8": lambda s: [moe.moe_grouped_dgrad_fp8(
        dev(4, 128), dev(1, 128, 128, dtype=U8), dev(1, 1, 1, dtype=F32), dev(2, dtype=I32),
        stream=s)],
    "moe_combine": lambda s: [moe.moe_combine(dev(8, 128), dev(4, 2, dtype=F32), dev(4, 2, dtype=I32),
                                              -1, stream=s)],
    "moe_seq_balance_loss": lambda s: [moe.moe_seq_balance_loss(
        dev(4, 2, dtype=I32), dev(4, 2, dtype=F32), dev(2, dtype=I32), 16, stream=s)],
    "moe_probe_fp8_mfma": lambda s: [moe.moe_probe_fp8_mfma(1, 1, stream=s)[0]],
    "moe_probe_hbm": lambda s: [moe.moe_probe_hbm(0, dev(64, dtype=I32), stream=s)],
    "moe_block_norm": lambda s: moe.moe_block_norm(dev(4, 16), dev(4, 16), dev(16, dtype=F32),
                                                   dev(16, dtype=F32), stream=s),
    **{f"moe_block_norm_backward {k}": lambda s, g=g: moe.moe_block_norm_backward(
        dev(4, 16), dev(4, 16), dev(4, 16), dev(4, 16), dev(16, dtype=F32), dev(16, dtype=F32), g(),
        stream=s)
       for k, g in {"channel": lambda: dev(16, dtype=F32), "full": lambda: dev(4, 16)}.items()},
    "moe_grouped_gemm_bf16": lambda s: [moe.moe_grouped_gemm_bf16(
        dev(4, 16), dev(1, 8, 16), dev(2, dtype=I32), 4, stream=s)],
    "moe_grouped_wgrad_bf16": lambda s: [moe.moe_grouped_wgrad_bf16(
        dev(4, 16), dev(4, 8), dev(2, dtype=I32), 4, stream=s)],
    "moe_swiglu": lambda s: [moe.moe_swiglu(dev(4, 16), stream=s)],
    "moe_swiglu_backward": lambda s: moe.moe_swiglu_backward(dev(4, 16), dev(4, 8), stream=s),
    "moe_grad_norm": lambda s: moe.moe_grad_norm(moe.GradList([dev(8)]), stream=s),
    "moe_grad_scale": lambda s: [moe.moe_grad_scale(moe.GradList([dev(8)]),
                                                    dev(1, dtype=torch.float64), 1.0, stream=s)],
    "moe_grad_clip": lambda s: [moe.moe_grad_clip(moe.GradList([dev(8)]), 1.0, stream=s)],
}


@pytest.fixture
def world(monkeypatch):
    """(the caller's stream, list of (stream, tensor) for every allocation)."""
    home = Stream()
    now, made = [home], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    def maker(real):
        def make(*shape, **kw):
            kw.pop("device", None)
            t = real(*shape, **kw).as_subclass(Device)
            made.append((now[-1], t))
            return t
        return make

    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, maker(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(moe, "_queue", lambda s: (s or now[-1]).cuda_stream)
    monkeypatch.setattr(moe, "lib", Library)
    make_list = moe.GradList.__init__

    def make_list_before(self, *a):         # the program's own, not the call's
        make_list(self, *a)
        made.clear()

    monkeypatch.setattr(moe.GradList, "__init__", make_list_before)
    return home, made


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_belongs_to_its_stream(world, name):
    home, made = world
    stream = Stream()
    results = {id(t) for t in CALLS[name](stream) if t is not None}
    assert made and all(s is stream for s, _ in made)
    # the caller reads the results on its own stream, and may drop them there
    for _, t in made:
        if id(t) in results:
            assert t.users == [home]


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_without_a_stream_is_the_current_streams(world, name):
    home, made = world
    CALLS[name](None)
    assert made and all(s is home and t.users is None for s, t in made)


@pytest.mark.parametrize("name", ["moe_grad_norm", "moe_grad_scale", "moe_grad_clip"])
def test_a_list_dropped_behind_a_call_keeps_its_table_until_the_call_has_run(world, monkeypatch, name):
    home, made = world
    lists = []
    make_list = moe.GradList.__init__

    def note(self, *a):
        make_list(self, *a)
        self.table, self.ws = (t.as_subclass(Device) for t in (self.table, self.ws))
        lists.append(self)

    monkeypatch.setattr(moe.GradList, "__init__", note)
    stream = Stream()
    CALLS[name](stream)
    CALLS[name](None)
    CALLS[name](home)
    other, own, named = lists
    for held in ("table", "ws"):
        assert getattr(other, held).users == [stream]
        assert getattr(own, held).users is None and getattr(named, held).users is None
    monkeypatch.setattr(moe, "GradList", lambda tensors: own)
    with torch.cuda.stream(stream):     # the current stream of the call, not of the list
        CALLS[name](None)
    assert own.table.users == own.ws.users == [stream]
