"""Host threads that call the page operations at the same time, each with a cache of its own."""
import threading

import pytest
import torch

import exact_attention_103_b200 as ea

pytestmark = pytest.mark.gpu


def test_caches_of_different_sizes():
    """Requests and slots lie in shared memory of the call's own size: one thread's does not bound another's."""
    errors = []

    def work(slots):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                c = ea.KVCache.empty(1, 64, 16, 1, 64, slots, 1)
                all_slots = torch.arange(slots, device="cuda", dtype=torch.int32)
                none = torch.zeros(slots, device="cuda", dtype=torch.int32)
                for _ in range(1500):
                    c.alloc(all_slots, none)
            s.synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the test's own thread)
            errors.append(e)
    threads = [threading.Thread(target=work, args=(n,)) for n in (8192, 2900, 8000, 3500)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    ea.get_device_status()
