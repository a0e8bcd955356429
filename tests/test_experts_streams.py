"""Whose memory and which device the calls of expert layers and 4-bit weights use, without a GPU."""
import contextlib
import types

import pytest
import torch

import decode_gemm_bf16_b200 as uw


class _Seen(torch.Tensor):
    """A tensor that notes the streams it is recorded on."""

    def record_stream(self, stream):
        self.streams = getattr(self, "streams", []) + [stream]


def _seen():
    return torch.zeros(4, 32, dtype=torch.uint8).as_subclass(_Seen)


def _matrix():
    m = uw.MxMatrix.__new__(uw.MxMatrix)
    m._hold(_seen(), _seen(), (4, 64))
    return m


def test_inputs_are_recorded_on_a_given_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    device = torch.device("cuda", 0)
    s = types.SimpleNamespace(cuda_stream=77, device=device)
    t, m = _seen(), _matrix()
    assert uw._run(device, s, lambda handle, *a: (handle, len(a)), t, m, None, (1, 2), True) == (77, 5)
    assert t.streams == m.codes.streams == m.scales.streams == [s]


def test_a_stream_of_another_device_is_refused():
    s = types.SimpleNamespace(cuda_stream=77, device=torch.device("cuda", 1))
    t = _seen()
    with pytest.raises(ValueError):
        uw._run(torch.device("cuda", 0), s, lambda *a: None, t)
    assert not hasattr(t, "streams")


def test_workspace_is_sized_for_the_weights_device(monkeypatch):
    current = []

    @contextlib.contextmanager
    def device(d):
        current.append(torch.device(d))
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    seen = []
    monkeypatch.setattr(uw, "_group_bytes", lambda a: seen.append(list(current)) or 512)
    m = _matrix()
    m.device = torch.device("cuda", 1)
    assert uw.uw_gemm_grouped_workspace(6, m) == 512 and seen == [[torch.device("cuda", 1)]]


def _calls():
    """name -> (inputs, call(inputs, stream)): every entry point that takes a stream."""
    from tests.test_gpu_experts_exact import _offsets, _rows, _weights
    X, W = _rows(64, 512, 1), _weights(4, 128, 512, 2)
    Wm, off = uw.uw_mx_quantize(W), _offsets([20, 0, 30, 14])
    copy = lambda m: uw.MxMatrix(m.codes.clone(), m.scales.clone())  # noqa: E731
    rows = torch.arange(63, -1, -1, device="cuda").int()
    pos = torch.arange(64, device="cuda").int().view(32, 2)
    one = uw.uw_mx_quantize(W[0])
    return {
        "quantize": (lambda: [X.clone()], lambda a, s: uw.uw_mx_quantize(a[0], stream=s).codes),
        "dequantize": (lambda: [copy(Wm)], lambda a, s: uw.uw_mx_dequantize(a[0], stream=s)),
        "mx_gemm": (lambda: [X.clone(), copy(one)], lambda a, s: uw.uw_mx_gemm(a[0], a[1], stream=s)),
        "mx_gemm, strided": (lambda: [X.t().contiguous().t(), copy(one)], lambda a, s: uw.uw_mx_gemm(a[0], a[1], stream=s)),
        "route": (lambda: [X[:, :40].clone().float()], lambda a, s: uw.uw_route(a[0], 6, stream=s).weights),
        "grouped": (lambda: [X.clone(), W.clone(), off.clone(), rows.clone(), W.clone()],
                    lambda a, s: uw.uw_gemm_grouped(a[0], a[1], a[2], rows=a[3], up=a[4], stream=s)),
        "grouped, 4 bits": (lambda: [X.clone(), copy(Wm), off.clone(), rows.clone(), copy(Wm)],
                            lambda a, s: uw.uw_gemm_grouped(a[0], a[1], a[2], rows=a[3], up=a[4], stream=s)),
        "combine": (lambda: [X.clone(), pos.clone(), torch.ones(32, 2, device="cuda")],
                    lambda a, s: uw.uw_combine(a[0], a[1], a[2], stream=s)),
    }


@pytest.mark.gpu
def test_inputs_may_be_dropped_while_their_stream_is_busy():
    """A stream held up for some milliseconds: what its call will read is not given to others meanwhile."""
    s = torch.cuda.Stream()
    for name, (inputs, call) in _calls().items():
        a = inputs()
        torch.cuda.synchronize()
        want = call(a, None)
        sizes = [t.numel() * t.element_size() for x in a for t in ((x.codes, x.scales) if isinstance(x, uw.MxMatrix) else (x,))]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)      # about 10 ms
        got = call(a, s)
        del a
        over = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        s.synchronize()
        assert torch.equal(got, want), name
        torch.cuda.synchronize()
        del over
    assert uw.uw_last_device_status() == 0
