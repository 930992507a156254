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
