"""Stand-ins for CUDA tensors, streams and the library's calls, so that what
the Python front end does with them can be tested without a GPU: on which
stream and device a result is allocated, which tensors are held for which
stream, what is refused before anything is enqueued."""
import contextlib

import torch


class Stream:
    def __init__(self, raw, device=0):
        self.cuda_stream, self.device_index = raw, device
        self.device = torch.device("cuda", device)

    def __repr__(self):
        return f"Stream({self.cuda_stream})"


class Tensor:
    """What the front end asks of a tensor.  made_on: the raw stream that was current when it was allocated."""

    def __init__(self, shape, dtype=torch.float32, device=0, made_on=None, address=4096):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, True
        self.device, self.made_on, self.address = torch.device("cuda", device), made_on, address
        self.held_for = []

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return True

    def is_inference(self):
        return False

    def data_ptr(self):
        return self.address

    def record_stream(self, stream):
        self.held_for.append(stream.cuda_stream)

    def _part(self, shape):
        t = Tensor(shape, self.dtype, self.device.index, self.made_on, self.address)
        t.held_for = self.held_for   # the same memory
        return t

    def split(self, sizes):
        return [self._part((n,)) for n in sizes]

    def view(self, *shape):
        return self._part(shape[0] if len(shape) == 1 and isinstance(shape[0], tuple) else shape)

    def __getitem__(self, key):
        return self._part((key.stop - key.start,))


class Cuda:
    """Puts the stand-ins in place of torch's and the library's.  calls: (name, arguments) of each library call."""

    def __init__(self, monkeypatch, api):
        self.streams, self.calls, self.made, self.current_device = [Stream(0x10)], [], [], 0
        monkeypatch.setattr(torch, "empty", self.empty)
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.streams[-1])
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current_device)
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: Stream(raw))
        monkeypatch.setattr(torch.autograd.graph, "increment_version", lambda t: None)
        monkeypatch.setattr(api, "_current_stream", lambda device: self.streams[-1].cuda_stream)
        if hasattr(api, "_current_device"):
            monkeypatch.setattr(api, "_current_device", lambda: self.current_device)
        for name in ("ws_logprobs", "ws_logprobs_backward", "ws_distill", "ws_topk", "ws_topk_workspace_init", "ws_preprocess",
                     "ws_detect", "ws_detect_workspace_init"):
            monkeypatch.setattr(api.B, name, self.call(name))
        monkeypatch.setattr(api.B, "ws_topk_workspace_bytes", lambda *a: (0, 1000))
        monkeypatch.setattr(api.B, "ws_detect_workspace_bytes", lambda *a: (0, 1000))

    def empty(self, *shape, dtype=torch.float32, device="cuda"):
        if len(shape) == 1 and not isinstance(shape[0], int):
            shape = tuple(shape[0])
        index = torch.device(device).index or 0
        t = Tensor(shape, dtype, index, self.streams[-1].cuda_stream, address=1 << (20 + len(self.made)))
        self.made.append(t)
        return t

    @contextlib.contextmanager
    def stream(self, s):
        self.streams.append(s if s is not None else self.streams[-1])
        yield
        self.streams.pop()

    def call(self, name):
        def called(*args):
            self.calls.append((name, args))
            return 0
        return called
