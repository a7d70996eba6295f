"""Argument checks of the Python binding that need no device: tensors that only
claim to be on one stand in for device memory."""
import pytest
import torch

import mixed_gemm_amd as mg


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def claimed(t):
    return t.as_subclass(OnDevice)


def workspace(desc, M, host=None):
    """An Act whose buffers claim to be on the device, all but the one named `host`."""
    a = mg.Act.empty(desc, M, "cpu")
    for n in ("Aq", "As", "XO"):
        if n != host:
            setattr(a, n, claimed(getattr(a, n)))
    return a


@pytest.mark.parametrize("host", ["Aq", "As", "XO"])
def test_workspace_in_host_memory_is_refused(host):
    desc = mg.make_desc(64, 32, 4)
    with pytest.raises(ValueError, match="device tensor expected"):
        mg._act_struct(desc, workspace(desc, 5, host), 5)


def test_workspace_with_gaps_is_refused():
    desc = mg.make_desc(64, 32, 4)
    for n in ("Aq", "As", "XO"):
        a = workspace(desc, 5)
        t = getattr(a, n)
        setattr(a, n, claimed(torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]))
        with pytest.raises(ValueError, match="contiguous"):
            mg._act_struct(desc, a, 5)


def test_workspace_on_the_device_is_taken():
    for k in (4, 0):                     # k = 0: XO is empty
        desc = mg.make_desc(64, 32, k)
        a = workspace(desc, 5)
        c = mg._act_struct(desc, a, 5)
        assert c.Aq == a.Aq.data_ptr() and c.As == a.As.data_ptr() and c.XO == (a.XO.data_ptr() or None)
