"""Plans of batches of different sizes, called by several host threads at once."""
import threading

import pytest

pytestmark = pytest.mark.gpu


def test_threads():
    import torch
    import uncertainty_aware_delta_gb300 as kdn

    i32 = dict(dtype=torch.int32, device="cuda")
    call, failed = kdn.library().kdn_cache_plan, []

    def work(n, calls, go):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ctx, new, table = torch.zeros(n, **i32), torch.ones(n, **i32), torch.full((n, 1), -1, **i32)
                free, count, ws = torch.arange(n, **i32), torch.tensor([n], **i32), torch.empty(256, dtype=torch.uint8, device="cuda")
                out = kdn.kdn_cache_plan(ctx, new, table, free, count, page=16, capacity=n, workspace=ws)
                # the calls alone, side by side: the interpreter is not held while they run
                args = (n, 16, 1, n, n, *(t.data_ptr() for t in (ctx, new, table, free, count, *out, ws)), 256, stream.cuda_stream)
                go.wait()
                for i in range(calls):
                    st = call(*args)
                    if st:
                        failed.append((n, i, st))
                        return
                assert bool(out.granted.all()) and int(out.free_left) == 0 and kdn.kdn_read_device_status(ws, stream) == 0
        except Exception as e:  # noqa: BLE001
            failed.append((n, repr(e)))
            go.abort()

    sizes = (16000, 3, 9000, 1, 14000, 100)
    go = threading.Barrier(len(sizes))
    threads = [threading.Thread(target=work, args=(n, 5000, go)) for n in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
