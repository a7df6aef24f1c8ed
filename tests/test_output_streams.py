"""Which stream's memory a new output is taken from, on the CPU: torch's stream objects are stand-ins that record."""
import contextlib

import pytest
import torch

from token_dispatch_topk_b200 import binding as B


class Like:
    """A stand-in for a tensor on cuda:0; new_empty answers with the stream that was current."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self):
        self.current = "the current stream"

    def new_empty(self, shape, dtype):
        return self.current


@pytest.mark.parametrize("handle,want", [(None, "the current stream"), (0, ("default", 0)), (4096, ("external", 4096))])
def test_a_new_output_comes_from_the_memory_of_the_stream_that_writes_it(monkeypatch, handle, want):
    """Handle 0 is the default stream, whereas ExternalStream(0) is one of torch's pool streams."""
    like = Like()

    @contextlib.contextmanager
    def on(stream):
        before, like.current = like.current, stream
        yield
        like.current = before

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", torch.device(device).index))
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device: ("external", handle) if handle else ("pool", "any"))
    assert B._new(like, (4, 4), torch.uint8, handle) == want
