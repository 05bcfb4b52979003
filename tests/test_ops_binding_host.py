"""Checks of the operators' binding that need no device: sizes past the types
of the C entries, and streams of another device."""
import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from combine_symmetric_memory_amd import ops
    return ops


META = torch.device("meta")


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=META)


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5])
def test_sizes_past_int32_are_refused(ops, n):
    # ctypes would pass 2^32 + 5 on as 5
    for shape in ((n, 1), (1, n)):
        with pytest.raises(ValueError, match="int32"):
            ops._rows(_meta(*shape), META, "x")
        with pytest.raises(ValueError, match="int32"):
            ops._norm_desc(_meta(*shape), None, None, None, None, 1.0, 1e-6)
    i = _meta(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="int32"):
        ops._groups(i, i, 4, META)
    for kw in (dict(topk=n), dict(topk=2, groups=n), dict(topk=2, kept=n)):
        with pytest.raises(ValueError, match="int32"):
            ops._route_desc(8, kw.pop("topk"), "softmax", False, 1.0, **kw)


def test_the_largest_sizes_pass_the_binding(ops):
    n = 2 ** 31 - 1
    assert ops._rows(_meta(n, 1), META, "x") == 1
    assert ops._rows(_meta(1, n), META, "x") == n


def test_a_stream_of_another_device_is_refused(ops, monkeypatch):
    # made current, it would take the call to its own device's default stream
    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

    entered = []

    class Context:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            entered.append(self.what)

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    dev = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="stream"):
        with ops._Elsewhere(dev, Stream(1)):
            pass
    assert not entered
    s = Stream(0)
    with ops._Elsewhere(dev, s):
        assert entered == [dev, s]
