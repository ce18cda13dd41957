"""The paged cache's calls from several host threads at once, each with a stream and a workspace of
its own: first calls of a kernel among them (every thread may be the one that sets its limits)."""
import threading

import pytest
import torch

from tests.test_gpu_paged import Cache

pytestmark = pytest.mark.gpu


def test_threads(lib):
    # different kernels per head size, dtype and group; two threads to each
    kinds = [(8, 1, 64, "bf16"), (32, 2, 96, "bf16"), (2, 2, 256, "f32"), (12, 1, 72, "f32")] * 2
    caches = [Cache(lib, [700, 33, 300], nq, nkv, hd, 16, dt, seed=i)
              for i, (nq, nkv, hd, dt) in enumerate(kinds)]
    before = [c.score.clone() for c in caches]
    streams = [torch.cuda.Stream() for _ in caches]
    torch.cuda.synchronize()
    start, out, failed = threading.Barrier(len(caches)), [None] * len(caches), []

    def work(i):
        try:
            c = caches[i]
            start.wait(timeout=60)
            with torch.cuda.stream(streams[i]):
                out[i] = c.decode()
                ws = torch.empty(lib.tp_kv_evict_paged_workspace(c.desc, 200), dtype=torch.uint8,
                                 device=c.kp.device)
                new = torch.empty_like(c.lens)
                kept = c.score.clone()
                kp, vp = c.kp.clone(), c.vp.clone()
                lib.tp_kv_evict_paged(c.desc, kept, c.lens, 200, 20, kp, vp, c.tables, new, workspace=ws)
                out[i] += (new,)
            streams[i].synchronize()
        except BaseException as e:       # an exception in a thread fails the test, not the thread alone
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(caches))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for c, b, (o, lse, new) in zip(caches, before, out):
        c.check(o, lse, b)
        assert new.tolist() == [200, 33, 200]
    lib.tp_check_device_error()
