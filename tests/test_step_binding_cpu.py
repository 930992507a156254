"""The binding's objects of a decoding step, without a GPU."""
import threading
import time

import pytest

from lossless_bit_weight_02_amd import w12


@pytest.mark.parametrize("cls,names", [(w12.KVCache, ("k", "v", "k_scale", "v_scale")),
                                       (w12.KVBatch, ("table", "lens", "q_start", "positions", "tree"))])
def test_tensors_are_read_only(cls, names):
    """A tensor whose address the library has cannot be replaced unnoticed."""
    obj = object.__new__(cls)
    obj._tensors = {n: object() for n in names}
    for n in names:
        assert getattr(obj, n) is obj._tensors[n]
        with pytest.raises(AttributeError):
            setattr(obj, n, None)


def test_one_call_at_a_time(monkeypatch):
    """Calls that share a stream's scratch do not run into each other, one that fails lets the next one in."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(w12, "_step_buffers", {})
    inside, most, addresses = [0], [0], set()

    def launches(buf):
        inside[0] += 1
        most[0] = max(most[0], inside[0])
        addresses.add(buf)
        time.sleep(0.01)                    # (the interpreter's lock is free here, as in the library)
        inside[0] -= 1
        return w12.W12_OK

    def work():
        for _ in range(5):
            w12._step_call("attention", 1000, torch.device("cpu"), 0, launches)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert most[0] == 1 and len(addresses) == 1
    with pytest.raises(w12.W12Error):
        w12._step_call("attention", 1000, torch.device("cpu"), 0, lambda buf: w12.W12_ERR_ARG)
    work()


def test_output_apart_from_inputs():
    torch = pytest.importorskip("torch")
    buf = torch.zeros(1000, dtype=torch.bfloat16)
    out = buf[:64].view(4, 16)

    def check(at, m=4, cols=16, ld=16, size=2, same=False):
        w12._check_apart(out, "q", buf.data_ptr() + 2 * at, m, cols, ld, size, same)

    check(64)                                           # side by side
    check(0, same=True)                                 # the rows themselves
    check(0, m=1, ld=99, same=True)
    for bad in (dict(at=0), dict(at=0, ld=32, same=True), dict(at=8, same=True), dict(at=63), dict(at=0, size=4, same=True)):
        with pytest.raises(ValueError):
            check(**bad)
    out = buf[64:128].view(4, 16)
    check(0)
    with pytest.raises(ValueError):
        check(0, ld=17)
