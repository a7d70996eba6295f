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


def wrong(rows, cols):
    """Outputs that do not fit [rows][cols], with what the refusal says."""
    return [(on(rows + 1, cols), "must be"), (on(rows, cols + 32), "must be"), (on(rows, cols, dtype=torch.float16), "dtype"),
            (on(cols, rows).t(), "contiguous"), (torch.zeros(rows, cols), "device")]


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("i", range(5))
def test_linear_gradients_are_checked_first(nothing_runs, which, i):
    """An output that does not fit is refused before anything runs."""
    p, saved, dY, work = linear()
    out, says = wrong(*((M, K), (N, K))[which])[i]
    nothing_runs()
    for need in ((True, True), (which == 0, which == 1)):
        with pytest.raises(ValueError, match=says):
            mg.f8_backward(p, saved, dY, **{("dX", "dW")[which]: out}, work=work, need=need)


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("i", range(5))
def test_gated_gradients_are_checked_first(nothing_runs, which, i):
    ffn, saved, dY, work = gated()
    out, says = wrong(*((M, K), (F, K), (F, K), (N, F))[which])[i]
    nothing_runs()
    with pytest.raises(ValueError, match=says):
        mg.gated_ffn_backward(ffn, saved, dY, **{("dX", "dWg", "dWu", "dWd")[which]: out}, work=work)


def test_gated_weight_gradients_of_two_types(nothing_runs):
    ffn, saved, dY, work = gated()
    nothing_runs()
    with pytest.raises(ValueError, match="type"):
        mg.gated_ffn_backward(ffn, saved, dY, dWg=on(F, K), dWu=on(F, K, dtype=torch.bfloat16), work=work)


def test_gradients_of_no_rows_are_checked(nothing_runs):
    """Without rows the weight gradients are cleared: only ones that fit."""
    p, x, dY = mg.F8Plan(f8(N, K), f8(K, N)), f8(0, K), on(0, N)
    work = mg.F8Work(f8(0, N), f8(N, 32), f8(K, 32))
    ffn, saved = gated()[0], mg.GatedSaved(f8(0, K), f8(0, 512), f8(0, F))
    gwork = mg.GatedWork(f8(0, K), f8(0, F), on(0, dtype=torch.uint8), "e4m3", {})
    nothing_runs()
    for kw in (dict(dW=on(3, 3) + 1), dict(dX=on(1, K))):
        with pytest.raises(ValueError, match="must be"):
            mg.f8_backward(p, x, dY, work=work, **kw)
    for kw in (dict(dWg=on(3, 3)), dict(dWd=on(F, N)), dict(dX=on(1, K))):
        with pytest.raises(ValueError, match="must be"):
            mg.gated_ffn_backward(ffn, saved, dY, work=gwork, **kw)
    dW = on(N, K) + 1
    assert not mg.f8_backward(p, x, dY, dX=on(0, K), dW=dW, work=work)[1].any()


@pytest.mark.parametrize("name", ["gu", "h"])
def test_gated_saved_of_another_block(nothing_runs, name):
    ffn, saved, dY, work = gated()
    setattr(saved, name, f8(M, 256))
    nothing_runs()
    with pytest.raises(ValueError, match=f"saved.{name}"):
        mg.gated_ffn_backward(ffn, saved, dY, work=work)


@pytest.mark.parametrize("name,cols", [("x", K), ("gu", 512), ("h", F)])
def test_gated_saved_in_another_format(nothing_runs, name, cols):
    ffn, saved, dY, work = gated()
    setattr(saved, name, f8(M, cols, "e5m2"))
    nothing_runs()
    with pytest.raises(ValueError, match=f"saved.{name} must be e4m3"):
        mg.gated_ffn_backward(ffn, saved, dY, work=work)


class On1(On0):
    """A host tensor that says it is on device 1."""

    def get_device(self):
        return 1


def far(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(On1)


EPILOGUES = {
    "bias": lambda: mg.Epilogue(bias=far(N)),
    "residual": lambda: mg.Epilogue(residual=far(M, N)),
    "gate": lambda: mg.Epilogue(gate=mg.Mod(gate=far(1, N))),
    "gate index": lambda: mg.Epilogue(gate=mg.Mod(gate=on(2, N), index=far(M, dtype=torch.int32))),
    "gate index alone": lambda: mg.Epilogue(gate=mg.Mod(rows=2, index=far(M, dtype=torch.int32))),
    "one of several": lambda: mg.Epilogue(bias=on(N), gate=mg.Mod(gate=on(1, N)), residual=far(M, N)),
}


@pytest.mark.parametrize("kind", sorted(EPILOGUES))
def test_epilogue_on_another_device(nothing_runs, kind):
    """Kernels run on the current device and would read what the epilogue points at."""
    ep = EPILOGUES[kind]()
    p, x, ffn, work = mg.F8Plan(f8(N, K)), f8(M, K), *(gated()[i] for i in (0, 3))
    nothing_runs()
    for call in (lambda: mg.mg_f8_gemm(x, p.w, ep, on(M, N)), lambda: mg.f8_forward(p, on(M, K), ep, x, on(M, N)),
                 lambda: mg.gated_ffn_forward(ffn, on(M, K), Y=on(M, N), work=work, ep=ep)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_epilogue_on_the_current_device(nothing_runs):
    ep = mg.Epilogue(on(N), "silu", mg.Mod(gate=on(2, N), index=on(M, dtype=torch.int32)), on(M, N))
    p, x = mg.F8Plan(f8(N, K)), f8(M, K)
    nothing_runs()
    with pytest.raises(AssertionError, match="went through"):
        mg.mg_f8_gemm(x, p.w, ep, on(M, N))
