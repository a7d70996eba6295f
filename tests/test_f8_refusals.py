"""What the 8-bit layers' helpers refuse, on the CPU: host tensors that say they are
on device 0 stand for device tensors, and a call that reaches the library fails the test."""
import pytest
import torch

import mixed_gemm_amd as mg


class On0(torch.Tensor):
    """A host tensor that says it is on device 0."""
    is_cuda = True

    def get_device(self):
        return 0


def on(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(On0)


def f8(rows, cols, fmt="e4m3"):
    q, s = mg.mg_f8_bytes(rows, cols)
    return mg.F8(rows, cols, on(q, dtype=torch.uint8), on(s // 4, dtype=torch.int32), fmt)


M, K, N, F = 4, 64, 96, 160


def linear(fmt="e4m3"):
    """A plan, a checkpoint, a gradient and a workspace."""
    return (mg.F8Plan(f8(N, K), f8(K, N)), f8(M, K), on(M, N),
            mg.F8Work(f8(M, N, fmt), f8(N, 32, fmt), f8(K, 32)))


def gated(fmt="e4m3"):
    ffn = mg.GatedFFN(K, F, N, "silu", f8(512, K), f8(N, F), f8(K, 512), f8(F, N))
    back = {"dy": f8(M, N, fmt), "dyt": f8(N, 32, fmt), "ht": f8(F, 32), "dgu": f8(M, 512, fmt), "dgut": f8(512, 32, fmt),
            "xt": f8(K, 32)}
    work = mg.GatedWork(f8(M, K), f8(M, F), on(1 << 16, dtype=torch.uint8), fmt, back)
    return ffn, mg.GatedSaved(f8(M, K), f8(M, 512), f8(M, F)), on(M, N), work


@pytest.fixture
def nothing_runs(monkeypatch):
    """To be called once the operands are made."""
    def arm():
        def called():
            raise AssertionError("a call went through to the library")
        monkeypatch.setattr(mg, "_device", lambda: 0)
        monkeypatch.setattr(mg, "lib", called)
    return arm


@pytest.mark.parametrize("fmt,other", [("e4m3", "e5m2"), ("e5m2", "e4m3")])
def test_format_beside_a_workspace_of_the_other(nothing_runs, fmt, other):
    """A gradient format that the workspace does not have is refused, not ignored."""
    p, saved, dY, work = linear(fmt)
    ffn, kept, dy, gwork = gated(fmt)
    nothing_runs()
    with pytest.raises(ValueError, match=other):
        mg.f8_backward(p, saved, dY, fmt=other, work=work)
    with pytest.raises(ValueError, match=other):
        mg.gated_ffn_backward(ffn, kept, dy, fmt=other, work=gwork)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("given", [False, True])
def test_the_workspace_has_the_format(nothing_runs, fmt, given):
    """Either format of the workspace, named again or not, reaches the library."""
    p, saved, dY, work = linear(fmt)
    ffn, kept, dy, gwork = gated(fmt)
    kw = {"fmt": fmt} if given else {}
    nothing_runs()
    with pytest.raises(AssertionError, match="went through"):
        mg.f8_backward(p, saved, dY, work=work, **kw)
    with pytest.raises(AssertionError, match="went through"):
        mg.gated_ffn_backward(ffn, kept, dy, work=gwork, **kw)
