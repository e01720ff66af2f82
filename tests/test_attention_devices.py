"""Which device and stream a call of the attention half runs on, on the CPU:
stand-ins for tensors that are on some cuda device, and for the library."""
import pytest
import torch

import moe_lora_expert_gb300 as m
from moe_lora_expert_gb300 import attention as A


class Stand:
    """What the binding asks of a contiguous tensor on cuda:index (-1: the CPU)."""

    def __init__(self, shape, dtype, index=1):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device, self.is_cuda = torch.device("cuda", index) if index >= 0 else torch.device("cpu"), index >= 0

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st) if i is None else st[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.used_on = stream

    def moved(self, index):
        return Stand(self.shape, self.dtype, index)


class Stream:
    def __init__(self, handle, index):
        self.cuda_stream, self.device_index = handle, index

    def synchronize(self):
        pass


@pytest.fixture
def fake(monkeypatch):
    """Stand-ins for the library's entry points and torch's devices: the calls
    (name, device that was current, stream), and the current device."""
    if A._rope_fn is None:
        A._bind()
    calls, current = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    for name in CALLS:
        monkeypatch.setattr(A, name, lambda args, handle, name=name: calls.append((name, current[0], handle)) or 0)
    monkeypatch.setattr(A, "_raw_stream", lambda index: 100 * index)
    monkeypatch.setattr(A, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(A, "_capturing", lambda: False)
    monkeypatch.setattr(A, "_captured_workspace", lambda index, handle: None)
    monkeypatch.setitem(A._workspaces, 1, {handle: (1 << 20, 1 << 30, None) for handle in (7, 100)})
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "zeros", lambda n, dtype, device: Stand((n,), dtype, device.index))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: Stream(0, index))
    return calls, current


def half(*shape):
    return Stand(shape, torch.bfloat16)


def ints(*shape):
    return Stand(shape, torch.int32)


def floats(*shape):
    return Stand(shape, torch.float32)


def cache_parts():
    return dict(k=Stand((10, 2, 16, 64), torch.uint8), v=Stand((10, 2, 16, 64), torch.uint8), k_scale=floats(10, 2),
                v_scale=floats(10, 2))


def cache():
    return m.PagedKVCache(**cache_parts())


CALLS = {
    "_rope_fn": (lambda **a: m.moe_rope(**a), dict(
        q=half(4, 8, 64), positions=ints(4), cos_sin=floats(9, 64), k=half(4, 2, 64), q_out=half(4, 8, 64),
        k_out=half(4, 2, 64), status=ints(4))),
    "_append_fn": (lambda **a: cache().append(**a), dict(
        k=half(4, 2, 64), v=half(4, 2, 64), block_table=ints(4, 8), seq_lens=ints(4), cu_q=ints(5), q=half(4, 8, 64),
        cos_sin=floats(9, 64), positions=ints(4), q_out=half(4, 8, 64))),
    "_attend_fn": (lambda **a: cache().attend(**a), dict(
        q=half(4, 8, 64), block_table=ints(4, 8), seq_lens=ints(4), cu_q=ints(5), out=half(4, 8, 64), lse=floats(4, 8))),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("now", [0, 1])
def test_calls_run_on_their_tensors_device(fake, name, now):
    """Tensors on cuda:1 while another device is current, and while it is."""
    calls, current = fake
    call, args = CALLS[name]
    current[0] = now
    call(**args)
    call(**args, stream=Stream(7, 1))
    assert calls == [(name, 1, 100), (name, 1, 7)] and current[0] == now


@pytest.mark.parametrize("name,operand", [(n, o) for n, (_, args) in CALLS.items() for o in args if (n, o) != ("_rope_fn", "q")])
@pytest.mark.parametrize("index", [0, -1])
def test_operands_are_on_one_device(fake, name, operand, index):
    """An operand that is elsewhere is refused by its name, before anything runs."""
    call, args = CALLS[name]
    with pytest.raises(ValueError, match=rf"\b{operand}\b"):
        call(**{**args, operand: args[operand].moved(index)})
    assert not fake[0]


def test_rope_takes_no_cpu_tensors(fake):
    call, args = CALLS["_rope_fn"]
    with pytest.raises(ValueError, match="q must be"):
        call(**{k: t.moved(-1) for k, t in args.items()})


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(fake, name):
    call, args = CALLS[name]
    with pytest.raises(ValueError, match="stream"):
        call(**args, stream=Stream(7, 0))
    assert not fake[0]


@pytest.mark.parametrize("part", ["v", "k_scale", "v_scale"])
def test_a_cache_is_on_one_device(fake, part):
    cache()
    parts = cache_parts()
    with pytest.raises(ValueError, match=part):
        m.PagedKVCache(**{**parts, part: parts[part].moved(0)})


@pytest.mark.parametrize("name", CALLS)
def test_operands_of_a_call_on_another_stream_are_kept(fake, name):
    """Their memory may not be handed out while that stream still uses it."""
    call, args = CALLS[name]
    args = {k: t.moved(1) for k, t in args.items()}
    call(**args)
    assert not any(hasattr(t, "used_on") for t in args.values())
    stream = Stream(7, 1)
    call(**args, stream=stream)
    assert all(t.used_on is stream for t in args.values())
