"""The wrappers' first calls from several threads at once: one of them loads the extension module and binds it."""
import threading
import time

from kalman_delta_rule_b200 import binding as B
from kalman_delta_rule_b200 import build


def test_one_thread_loads_the_module(monkeypatch):
    build.build()
    made = []

    class Module:
        bound = 0

        def bind(self, *addresses):
            time.sleep(0.05)
            self.bound = len(addresses)

        def raise_with(self, error):
            assert error is B.KdnError

    def slow(torch):
        made.append(Module())
        time.sleep(0.05)
        return made[-1]
    monkeypatch.setattr(B, "_native_module", slow)
    monkeypatch.setattr(B, "_cuda", lambda: None)
    monkeypatch.setattr(B, "_native_mod", None)
    got = []
    threads = [threading.Thread(target=lambda: got.append(B._native())) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and len(got) == 8 and all(m is made[0] and m.bound == 8 for m in got)
