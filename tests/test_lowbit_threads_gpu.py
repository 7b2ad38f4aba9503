"""Calls of the norm, the quantizer and the product from several Python threads."""
from __future__ import annotations

import ctypes
import subprocess
import threading
import time

import pytest
import torch

import swiglu_backward_int8_b200 as sdq
from swiglu_backward_int8_b200 import _lib, lowbit
from tests import test_lowbit_paths_gpu as paths

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_call_waits(tmp_path, monkeypatch):
    """The entries replaced by one that sleeps as a launch into a full queue does: the short way gives the
    interpreter's lock back meanwhile, for each of the five functions."""
    (tmp_path / "slow.c").write_text("#include <unistd.h>\nint slow(void) { usleep(100000); return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / "slow.c"), "-o", str(tmp_path / "slow.so")], check=True)
    lib = ctypes.CDLL(str(tmp_path / "slow.so"))
    slow, real = ctypes.cast(lib.slow, ctypes.c_void_p).value, _lib.entry_addresses()
    paths._calls()                                           # (torch's own set-up is done)
    rounds, stop = [0], threading.Event()

    def other():
        while not stop.is_set():
            rounds[0] += 1
            time.sleep(0.001)

    thread = threading.Thread(target=other)
    thread.start()
    made = 0
    try:
        lowbit._marshal.bind(*(real[2] if i == 2 else slow for i in range(6)))     # (2: the workspace's size)
        for name in paths.NAMES:
            f = getattr(lowbit._marshal, name)

            def counted(*args, f=f, name=name):
                nonlocal made
                before, t0 = rounds[0], time.perf_counter()
                status = f(*args)
                if status == 0:
                    made += 1
                    # 100 rounds of a millisecond; with the lock held there is one at the most
                    assert time.perf_counter() - t0 >= 0.1 and rounds[0] - before >= 10, name
                return status

            monkeypatch.setattr(lowbit._marshal, name, counted)
        paths._calls()
    finally:
        stop.set()
        thread.join()
        lowbit._marshal.bind(*real)
    assert made == 8


def test_calls_from_threads_at_once():
    """Each thread on a stream of its own, with tensors of its own, gives what one thread gives."""
    want = paths._calls()
    failed = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = paths._calls()
                    for name in want:
                        for a, b in zip(got[name], want[name]):
                            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert sdq.sdq_device_status() == 0
