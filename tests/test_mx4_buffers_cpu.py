"""What the 4-bit experts hold is noted on every stream that reads it, once a stream;
host stand-ins for the tensors."""
from top_routing_grouped_fp32_gb300 import microscaling


class Buffer:
    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


def test_each_stream_is_noted_once():
    ex = object.__new__(microscaling.Mx4SwiGluExperts)
    ex.handle, ex._streams, ex._keep = None, set(), tuple(Buffer() for _ in range(4))
    for stream, raw in (("a", 17), ("b", 18), ("a", 17), ("b", 18)):
        ex._read_on(stream, raw)
    assert all(b.streams == ["a", "b"] for b in ex._keep)
