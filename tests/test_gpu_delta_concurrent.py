"""Every call of a delta-rule layer from several host threads at once, each on a stream and with
buffers of its own."""
import threading

import pytest

from test_gpu_delta_block import calls
from test_sequence_layers_ttt_amd import ttt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("long", [False, True])
def test_all_calls_in_host_threads(long):
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ttt.lib()
    dev = torch.device("cuda:0")
    sets = [calls(dev, long) for _ in range(4)]
    want = []
    for name, outs, fn in sets[0]:
        fn()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    bad = []

    def work(every):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                for (name, outs, fn), ref in zip(every, want):
                    fn()
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(outs, ref)):
                        bad.append(name)

    threads = [threading.Thread(target=work, args=(every,)) for every in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
