"""The handle of 4-bit weights, on host tensors: what it keeps and hands to the library."""
import copy
import io

import pytest
import torch

import routing_dispatch_expert_amd as moe


@pytest.fixture(autouse=True)
def _on_the_host(monkeypatch):
    """The handle's own checks want device tensors."""
    monkeypatch.setattr(moe, "_require", lambda *a: None)


def made(zero=True):
    """A handle of E = 2, N = 20, K = 136, group 64."""
    z = torch.randint(16, (2, 2, 4, 16), dtype=torch.uint8) if zero else None
    return moe.Q4Weights(torch.randint(256, (2, 2, 2, 1024), dtype=torch.uint8), torch.rand(2, 2, 4, 16).bfloat16(), z,
                         (2, 20, 136), 64, "u4")


def given(q):
    """A pointer to the struct that a call with q passes on."""
    return moe._q4(q)


def follows(q):
    s = given(q).contents
    assert s.codes == q.codes.data_ptr() and s.scale == q.scale.data_ptr()
    assert s.zero == (None if q.zero is None else q.zero.data_ptr())
    assert (s.kind, s.group) == (moe.Q4_KINDS[q.kind], q.group)


@pytest.mark.parametrize("zero", [True, False])
def test_struct_follows_the_tensors(zero):
    q = made(zero)
    follows(q)
    q.scale.mul_(2)   # in place: the same memory
    follows(q)


@pytest.mark.parametrize("name", ["codes", "scale", "zero", "shape", "group", "kind"])
def test_parts_are_not_exchanged(name):
    """No part can be replaced beside the address or size that the calls use."""
    q = made()
    value = getattr(q, name)
    other = value.clone() if isinstance(value, torch.Tensor) else value
    try:
        setattr(q, name, other)
    except AttributeError:
        pass
    follows(q)


def test_tensor_objects_of_others_do_not_matter():
    codes = torch.randint(256, (1, 1, 1, 1024), dtype=torch.uint8)
    q = moe.Q4Weights(codes, torch.rand(1, 1, 1, 16).bfloat16(), None, (1, 8, 8), 128, "u4")
    at = codes.data_ptr()
    codes.data = torch.zeros(8, dtype=torch.uint8)
    q.codes.data = torch.zeros(8, dtype=torch.uint8)
    assert given(q).contents.codes == at and tuple(q.codes.shape) == (1, 1, 1, 1024)


@pytest.mark.parametrize("how", ["deepcopy", "save"])
def test_copied_and_saved(how):
    q = made()
    if how == "deepcopy":
        r = copy.deepcopy(q)
    else:
        f = io.BytesIO()
        torch.save(q, f)
        f.seek(0)
        r = torch.load(f, weights_only=False)   # written just above
    for a, b in ((q.codes, r.codes), (q.scale, r.scale), (q.zero, r.zero)):
        assert torch.equal(a, b) and a.data_ptr() != b.data_ptr()
    assert (r.shape, r.group, r.kind) == (q.shape, q.group, q.kind)
    follows(r)


class _Host:
    """Stands for the device and stream of a call on host tensors."""
    stream, other = None, None

    def __init__(self, device, stream):
        pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        pass

    def empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype)

    def lent(self, t):
        return t


@pytest.mark.parametrize("workspace", [None, torch.empty(1, dtype=torch.uint8), torch.empty(1 << 20, dtype=torch.uint8),
                                       torch.empty(1, dtype=torch.uint8).expand(1 << 20),
                                       torch.empty(1 << 20, dtype=torch.uint8)[::4096].expand(4096, 256).t()],
                         ids=["none", "small", "large", "one byte expanded", "strided"])
def test_workspace_has_the_bytes_it_is_passed_for(workspace, monkeypatch):
    """What reaches the kernels as a workspace is one block of at least the size needed, whatever is lent."""
    passed = {}
    monkeypatch.setattr(moe, "_On", _Host)
    monkeypatch.setattr(moe, "moe_q4_matvec", lambda *a: passed.update(ws=a[9], n=a[10]))
    try:
        moe.matvec_q4(torch.zeros(3, 136), made(), workspace=workspace)
    except ValueError as e:
        assert "workspace" in str(e) and not workspace.is_contiguous()
        return
    ws, n = passed["ws"], passed["n"]
    assert n == moe.moe_q4_matvec_workspace_size(3, 136, "f32") > 0
    assert ws.untyped_storage().nbytes() - ws.storage_offset() * ws.element_size() >= n
    if workspace is not None and workspace.numel() >= n:
        assert ws is workspace


class _Stream:
    def __init__(self, index, cuda_stream):
        self.device, self.cuda_stream = torch.device("cuda", index), cuda_stream


def test_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream(1, 16))
    device = torch.device("cuda", 1)
    assert moe._On(device, None).stream.cuda_stream == 16
    on = moe._On(device, _Stream(1, 32))
    assert on.stream is on.other and on.stream.cuda_stream == 32
    assert moe._On(device, _Stream(1, 16)).other is None
    with pytest.raises(ValueError, match="stream"):
        moe._On(device, _Stream(0, 32))
    with pytest.raises(ValueError, match="stream"):   # also where the handles happen to be equal (both null streams)
        moe._On(device, _Stream(0, 16))
