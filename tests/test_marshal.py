"""The compiled argument marshalling against the Python one: the same arguments
reach the library, the same ones are refused with the same words (no GPU
needed; the calls' results are the GPU tests' part)."""
import ctypes
import inspect

import pytest
import torch

from fp8_relu_mlp_b200 import _abi as A

CALLS = ["quantize_block", "weight_block_cache_refresh", "linear_fwd_block", "linear_block", "up_proj_block",
         "mlp_fwd_block", "norm_gate_fwd", "norm_gate_bwd"]
SIZES = {"M": 5, "K": 256, "N": 384, "d": 256, "h": 512, "rows_per_gate": 2}


@pytest.fixture
def both(monkeypatch):
    """Runs a call each way; the way is the argument."""
    monkeypatch.setattr(A, "_marshal", A._marshal)  # put back afterwards
    if A._marshal is None:
        A._find_marshal(torch)
    m = A._marshal
    if m is None:
        pytest.skip("the module is not built")

    def way(compiled):
        monkeypatch.setattr(A, "_marshal", m if compiled else None)
    yield way


def arguments(name, value):
    """Sizes by name, 1e-6 for eps, value(i) for the i-th pointer."""
    out = {}
    for i, p in enumerate(inspect.signature(getattr(A, "fp8mlp_" + name)).parameters):
        out[p] = SIZES[p] if p in SIZES else 1e-6 if p == "eps" else value(i)
    return out


@pytest.mark.parametrize("name", CALLS)
def test_arguments_arrive_in_order(name, both, monkeypatch):
    full, seen = "fp8mlp_" + name, []
    args = arguments(name, lambda i: 0x10000 * (i + 1))
    both(True)
    m = A._marshal
    types = A._SIGS[full]

    def record(*a):
        seen.append(a)
        return A.OK
    fake = ctypes.CFUNCTYPE(ctypes.c_int, *types)(record)
    m.bind(full, ctypes.cast(fake, ctypes.c_void_p).value)
    try:
        getattr(A, full)(**args)
    finally:
        m.bind(full, ctypes.cast(getattr(A.lib, full), ctypes.c_void_p).value)
    both(False)
    monkeypatch.setattr(A, "_call", lambda n, *a: seen.append(a))
    getattr(A, full)(**args)
    as32 = lambda a: tuple(ctypes.c_float(v).value if isinstance(v, float) else v for v in a)  # noqa: E731
    assert len(seen) == 2 and as32(seen[0]) == as32(seen[1])


def outcome(fn, *args, **kw):
    try:
        return fn(*args, **kw)
    except Exception as e:
        return type(e), str(e)


class NoTensor:
    pass


@pytest.mark.parametrize("name", CALLS)
def test_the_same_refusals(name, both):
    fn = getattr(A, "fp8mlp_" + name)
    args = arguments(name, lambda i: 0x10000)
    big = torch.zeros(1 << 20)
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    bad = [big, big[::2], big.to(dev)[:0], torch.zeros(2, dtype=torch.uint8, device=dev)[1:], NoTensor(), "x", 1.5, True]
    pointers = [k for k, v in args.items() if v == 0x10000 and k != "stream"]
    for k in pointers:
        for v in bad:
            got = []
            for way in (True, False):
                both(way)
                got.append(outcome(fn, **{**args, "stream": 0, k: v}))
            assert got[0] == got[1], (k, v)
            assert got[0][0] in (ValueError, TypeError), (k, v)


@pytest.mark.parametrize("name", CALLS)
def test_streams_and_sizes(name, both):
    fn = getattr(A, "fp8mlp_" + name)
    args = arguments(name, lambda i: 0x10002)  # no address of these is aligned

    class Stream:
        cuda_stream = 0
    for change in [dict(stream=Stream()), dict(stream=0), dict(stream=NoTensor()), dict(stream="0")]:
        got = []
        for way in (True, False):
            both(way)
            got.append(outcome(fn, **{**args, **change}))
        assert got[0] == got[1], change
        assert got[0][0] is (A.Fp8MlpError if "NoTensor" not in str(change) and change["stream"] != "0" else AttributeError)
    both(True)
    first = next(iter(args))
    for v in (1 << 31, -(1 << 31) - 1, 1 << 70):
        with pytest.raises(OverflowError):
            fn(**{**args, first: v, "stream": 0})
    for v in ("1", None, 1.0):
        with pytest.raises(TypeError):
            fn(**{**args, first: v, "stream": 0})


def test_the_module_by_itself(both):
    both(True)
    m = A._marshal
    with pytest.raises(TypeError, match="6 arguments"):
        m.quantize_block(1, 2)
    with pytest.raises(KeyError):
        m.bind("fp8mlp_version", 1)
    with pytest.raises(KeyError):
        m.bind("fp8mlp_quantize_block", 0)  # NULL stays unbound
    assert set(m.names()) <= set(A.header_symbols())


def test_another_torch_is_left_alone(both, monkeypatch):
    class Torch:
        __version__ = "0.0.1"
    both(False)
    A._find_marshal(Torch)
    assert A._marshal is None


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("v", [1 << 70, 1 << 64, -(1 << 63) - 1])
def test_addresses_beyond_64_bits_are_refused(name, v, both):
    fn = getattr(A, "fp8mlp_" + name)
    args = arguments(name, lambda i: 0x10000)

    class Stream:
        cuda_stream = v
    pointers = [k for k, a in args.items() if a == 0x10000 and k != "stream"]
    for change in [dict(stream=v), dict(stream=Stream())] + [{k: v} for k in pointers]:
        got = []
        for way in (True, False):
            both(way)
            got.append(outcome(fn, **{**args, "stream": 0, **change}))
        assert got[0] == got[1] and got[0][0] is OverflowError, change
        assert got[0][1].startswith(next(iter(change)))
