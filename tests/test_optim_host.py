"""The optimizer's and the block-scaled stack's host side without a GPU: what is
kept alive, and what waits for what.  The library's calls are recorded, not
made."""
import gc
import weakref

import pytest
import torch

from fp8_relu_mlp_b200 import _abi as A
from fp8_relu_mlp_b200._order import as_stream
from fp8_relu_mlp_b200.block import BlockScaledStack
from fp8_relu_mlp_b200.optim import AdamW


class Stream:
    """Stands in for torch.cuda.Stream."""

    def __init__(self, log, handle):
        self.log, self.cuda_stream = log, handle

    def wait_stream(self, other):
        self.log.append(("wait", (self.cuda_stream, other.cuda_stream)))

    def synchronize(self):
        self.log.append(("sync", (self.cuda_stream,)))


@pytest.fixture
def calls(monkeypatch):
    """Library calls by name, with waits between them."""
    log = []
    for name in A._SIGS:
        if hasattr(A, name):
            monkeypatch.setattr(A, name, lambda *a, _n=name, **k: log.append((_n, a)))
    monkeypatch.setattr(A, "fp8mlp_norm_gate_bwd_workspace_size", lambda *a: 16)
    monkeypatch.setattr(A, "adamw_tensor", lambda n, *a: A.AdamwTensor(n=n))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(log, 1))
    return log


def parameter(n):
    return dict(grad=torch.zeros(n), master=torch.zeros(n))


@pytest.mark.parametrize("own", [False, True])
def test_a_workspace_outlives_the_steps_that_use_it(calls, own):
    # a step under way, or captured, holds the workspace's address: a larger plan must not free it
    opt = AdamW(max_norm=1.0, device="cpu", stream=Stream(calls, 2) if own else None)
    opt.add(**parameter(100))
    opt.step()
    first = weakref.ref(opt._workspace)
    opt.add(**parameter(1 << 18))
    opt.step()
    gc.collect()
    assert first() is not None and opt._workspace.numel() >= 17 * 8
    used = [a[3] for n, a in calls if n == "fp8mlp_grad_norm"]
    assert [w.numel() for w in used] == [16, 17 * 8]
    # they double, and a plan that fits takes the one there is
    for outgrown in (2, 2, 2):
        opt.add(**parameter(5))
        opt.step()
        assert len(opt._outgrown) == outgrown and opt._workspace.numel() == 2 * 17 * 8


def test_a_step_waits_for_the_current_stream(calls):
    opt = AdamW(max_norm=1.0, device="cpu", stream=Stream(calls, 2))
    opt.add(**parameter(100))
    for _ in range(2):
        del calls[:]
        opt.step()
        assert [c[0] for c in calls] == ["wait", "fp8mlp_grad_norm", "fp8mlp_adamw_step"] and calls[0] == ("wait", (2, 1))
    # in a capture the current stream is the optimizer's own: nothing to wait for, and no host wait that would end it
    opt.stream = Stream(calls, 1)
    opt.add(**parameter(100))
    del calls[:]
    opt.step()
    assert [c[0] for c in calls] == ["fp8mlp_grad_norm", "fp8mlp_adamw_step"]


def test_without_a_stream_nothing_waits(calls):
    opt = AdamW(device="cpu")
    opt.add(**parameter(100))
    opt.step()
    opt.set_lr(0.5)
    opt.read_state()
    assert [c[0] for c in calls] == ["fp8mlp_adamw_state_init", "fp8mlp_adamw_step"]


def test_the_stack_waits_for_its_fills_and_inputs(calls):
    net = BlockScaledStack(2, 4, 32, 64, device="cpu", stream=Stream(calls, 2))
    opt = None
    for call in (net.refresh_caches, net.forward, net.backward, lambda: net.train_step(opt)):
        del calls[:]
        call()
        assert calls[0] == ("wait", (2, 1)) and calls[1][0].startswith("fp8mlp_")
        if opt is None:
            del calls[:]
            opt = net.optimizer()
            # the weights are read on the current stream, behind steps that may still write them
            assert calls[0] == ("wait", (1, 2))
    net = BlockScaledStack(2, 4, 32, 64, device="cpu")
    del calls[:]
    net.train_step(net.optimizer())
    assert not [c for c in calls if c[0] in ("wait", "sync")]


def test_tensors_that_overlap_are_refused(calls):
    opt = AdamW(device="cpu")
    flat = torch.zeros(10000)
    opt.add(flat[:1000], master=flat[2000:3000])
    opt.add(flat[1000:2000], master=flat[3000:4000])  # side by side
    whole = flat[4000:9000]
    for grad, master in ((whole[:500], flat[3999:4499]),  # by one element
                         (flat[500:1500], whole[:1000]), (whole[:1000], whole[900:1900]), (whole[:1000], whole[:1000]),
                         (flat[:10000], torch.zeros(10000)), (flat[10:20], whole[:10])):
        with pytest.raises(ValueError, match="overlap"):
            opt.add(grad, master=master)
    with pytest.raises(ValueError, match="overlap"):
        opt.add(whole[:100], master=whole[100:200], state=dict(m=whole[200:300], v=whole[250:350]))
    with pytest.raises(ValueError, match="overlap"):
        opt.add(whole[:100], master=whole[100:200], weight=whole[200:250].view(torch.bfloat16),
                state=dict(m=whole[249:349], v=whole[400:500]))
    # what was refused left nothing behind
    assert len(opt.entries) == len(opt._descriptors) == 2
    opt.add(whole[:100], master=whole[100:200], weight=whole[200:250].view(torch.bfloat16),
            state=dict(m=whole[250:350], v=whole[400:500]))
    opt.add(flat[:0], master=flat[:0])


@pytest.mark.parametrize("bits,moments,scales", [
    (8, torch.float8_e5m2, torch.float32), (8, torch.int8, torch.float32), (8, torch.bool, torch.float32),
    (8, torch.float8_e4m3fn, torch.float64), (8, torch.uint8, torch.int32), (8, torch.uint8, None),
    (32, torch.int32, None), (32, torch.float64, None), (32, torch.float8_e4m3fn, None)])
@pytest.mark.parametrize("both", [False, True])
def test_states_of_another_type_are_refused(calls, bits, moments, scales, both):
    right = torch.float32 if bits == 32 else torch.float8_e4m3fn
    opt = AdamW(state_bits=bits, device="cpu")
    wrong = dict(m=torch.zeros(256, dtype=moments), v=torch.zeros(256, dtype=moments if both else right))
    if scales is not None:
        wrong.update(m_scale=torch.ones(2, dtype=scales if both else torch.float32), v_scale=torch.ones(2, dtype=scales))
    with pytest.raises(ValueError, match="moments must|m_scale"):
        opt.add(**parameter(256), state=wrong)
    good = {k: torch.zeros(256, dtype=right) for k in ("m", "v")}
    if bits == 8:
        good.update({k: torch.ones(2) for k in ("m_scale", "v_scale")})
        good["m"] = good["m"].view(torch.uint8)
    opt.add(**parameter(256), state=good)


@pytest.mark.parametrize("lr", [float("nan"), float("inf"), -float("inf")])
def test_a_rate_that_is_not_finite_is_refused(calls, lr):
    opt = AdamW(device="cpu")
    opt.set_lr(0.25)
    with pytest.raises(ValueError, match="finite"):
        opt.set_lr(lr)
    assert opt.read_state()["lr"] == 0.25


def test_streams_of_other_kinds(monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, d: made.append((h, d)) or "external")

    class Handle:
        cuda_stream = 77
    assert as_stream(5, "cuda:0") == "external" and as_stream(Handle(), "cuda:0") == "external"
    assert made == [(5, "cuda:0"), (77, "cuda:0")]
    own = Stream([], 3)
    assert as_stream(own, "cuda:0") is own
