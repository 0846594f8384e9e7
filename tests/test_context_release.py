"""A dropped context on the CPU: its finaliser makes no call, since the garbage collector may run it while a stream is
being captured; the next create or destroy releases what has gathered."""
import ctypes
import gc

import pytest

pytest.importorskip("torch")

import loss_scaled_adamw_gb300 as tl
from loss_scaled_adamw_gb300 import losses


class FakeLibrary:
    """Records which handles are destroyed, and refuses to create."""

    def __init__(self):
        self.destroyed = []

    def _destroy(self, handle):
        self.destroyed.append(handle.value)
        return tl.TL_OK

    tl_destroy = tl_loss_destroy = _destroy

    def tl_create(self, *args):
        return tl.TL_EINVAL

    tl_loss_create = tl_create

    def tl_status_string(self, rc):
        return b"refused"


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLibrary()
    monkeypatch.setattr(tl, "_lib", lib)
    monkeypatch.setattr(losses, "_lib", lib)
    yield lib
    tl._release_dropped()


def optimizer(handle):
    return tl.Context(ctypes.c_void_p(handle), [])


def objectives(handle):
    return losses.LossContext(ctypes.c_void_p(handle), 0)


@pytest.mark.parametrize("make", [optimizer, objectives])
def test_a_finaliser_makes_no_call(fake, make):
    ctx = make(5)
    del ctx
    cycle = [make(6)]
    cycle.append(cycle)
    del cycle
    gc.collect()
    assert fake.destroyed == []
    tl.tl_destroy(optimizer(7))
    assert sorted(fake.destroyed) == [5, 6, 7]


@pytest.mark.parametrize("make", [optimizer, objectives])
def test_the_next_create_or_destroy_releases(fake, make):
    null = ctypes.c_void_p()
    for handle, release in enumerate((lambda: tl.tl_destroy(optimizer(100)), lambda: tl.tl_loss_destroy(objectives(101)),
                                      lambda: tl.tl_create([], [], [], [], [], [], tl.make_config(), null),
                                      lambda: tl.tl_loss_create(1, stream=null)), 1):
        ctx = make(handle)
        del ctx
        assert handle not in fake.destroyed
        try:
            release()
        except tl.TLError as e:
            assert e.args
        assert fake.destroyed.count(handle) == 1


@pytest.mark.parametrize("make,destroy", [(optimizer, tl.tl_destroy), (objectives, tl.tl_loss_destroy)])
def test_a_destroyed_context_is_not_released_again(fake, make, destroy):
    ctx = make(9)
    destroy(ctx)
    destroy(ctx)
    del ctx
    gc.collect()
    tl._release_dropped()
    assert fake.destroyed == [9]
