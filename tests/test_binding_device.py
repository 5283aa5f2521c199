"""The block and optimizer calls run on their tensors' device, whichever is current: a launch, and the
code of a block, go to the current one.  On the CPU, with a library and tensors that only record."""
import contextlib
import types

import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg

torch = pytest.importorskip("torch")


class Fake:
    """A contiguous tensor on device 1, as far as the binding looks."""
    is_cuda = True
    device = torch.device("cuda", 1)

    def __init__(self, shape, dtype):
        self.shape, self.dtype = tuple(shape), dtype

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def stride(self):
        return (self.shape[1], 1)

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def element_size(self):
        return self.dtype.itemsize

    def new_empty(self, shape, dtype=None):
        return Fake((shape,) if isinstance(shape, int) else shape, dtype or self.dtype)


@pytest.fixture
def launches(monkeypatch):
    """[(entry point, the device that is current at its call)]"""
    seen, current = [], [0]
    real = cg.lib()

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        try:
            yield
        finally:
            current[0] = before

    class Library:
        def __getattr__(self, name):
            if name.endswith(("workspace_size", "_destroy")):
                return getattr(real, name)

            def call(*args):
                seen.append((name, current[0]))
                return 0
            return call
    blocks = cg.Block("4x0e", gate="channel", post_norm=True, next_norm=True), cg.AdamW([4, 3], "f32", 8)
    monkeypatch.setattr(cg, "lib", Library)
    monkeypatch.setattr(cg, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(cg, "_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(torch.cuda, "device", device)
    yield types.SimpleNamespace(seen=seen, block=blocks[0], opt=blocks[1], current=current)
    assert current == [0]


def test_every_call_runs_on_the_device_of_its_tensors(launches):
    b, o, f32 = launches.block, launches.opt, torch.float32
    rows, chan, stat = Fake((5, 4), f32), Fake((4,), f32), Fake((5,), f32)
    cg.norm_forward(b, rows, chan)
    cg.norm_backward(b, rows, chan, stat, rows)
    cg.join_forward(b, rows, rows, rows, chan, chan, chan)
    cg.join_backward(b, rows, rows, rows, rows, rows, chan, chan, chan, stat, stat)
    tensors = [Fake((4,), f32), Fake((3,), f32)]
    m, v = Fake((o.elements,), torch.int8), Fake((o.elements,), torch.uint8)
    scales, norm = Fake((2, o.blocks), f32), Fake((1,), torch.float64)
    schedule, flat = Fake((4,), torch.float64), Fake((o.elements,), f32)
    cg.grad_norm(o, tensors)
    cg.adamw_schedule(schedule, norm=norm)
    cg.adamw_step(o, tensors, tensors, m, v, scales, step=1, norm=norm)
    cg.adamw_state_read(o, m, v, scales)
    cg.adamw_state_write(o, flat, flat, m, v, scales)
    assert [name for name, _ in launches.seen] == [
        "cgtp_norm_forward", "cgtp_norm_backward", "cgtp_join_forward", "cgtp_join_backward", "cgtp_grad_norm",
        "cgtp_adamw_schedule_norm", "cgtp_adamw_step", "cgtp_adamw_state_read", "cgtp_adamw_state_write"]
    assert all(device == 1 for _, device in launches.seen), launches.seen


def test_tensors_may_come_from_a_generator(launches):
    """What the compiled calls do not take is listed again."""
    o, f32 = launches.opt, torch.float32
    m, v = Fake((o.elements,), torch.int8), Fake((o.elements,), torch.uint8)
    one = lambda: (Fake((n,), f32) for n in (4, 3))  # noqa: E731
    cg.grad_norm(o, one())
    cg.adamw_step(o, one(), one(), m, v, Fake((2, o.blocks), f32), step=1)
    assert [name for name, _ in launches.seen] == ["cgtp_grad_norm", "cgtp_adamw_step"]
