"""GPU: moe_paged_attention from several host threads on one stream, which share its scratch: the two launches of a call stay
together."""
import threading
import time

import pytest
import torch

from test_attention_ops import BF, Batch, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("side", [False, True])
def test_threads_on_one_stream(m, side):  # noqa: F811
    stream = torch.cuda.Stream() if side else torch.cuda.default_stream()
    batches = [Batch(60, [1, 2, 1], [9000, 500, 60], 2, 128, 16).fill(), Batch(61, [1] * 40, [700] * 40, 1, 128, 16).fill(),
               Batch(62, [3], [20011], 4, 128, 16).fill()]
    jobs = []
    for b, n_q in zip(batches, (8, 4, 16)):
        q = b.normal(b.T, n_q, 128).to(BF)
        call = lambda b=b, q=q, n=max(b.new): m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=n)  # noqa: E731
        with torch.cuda.stream(stream):
            jobs.append((call, call(), []))
    torch.cuda.synchronize()
    go = threading.Barrier(len(jobs))

    def work(call, want, outs):
        with torch.cuda.stream(stream):
            go.wait()
            for _ in range(200):
                outs.append(call())

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    m.moe_read_device_status()
    for _, want, outs in jobs:
        assert len(outs) == 200 and all(torch.equal(o, want) for o in outs)


def test_first_calls_of_two_threads_report_to_one_place(m, monkeypatch):  # noqa: F811
    made = m.Workspace

    class Slow(made):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            time.sleep(0.05)

    monkeypatch.setattr(m, "Workspace", Slow)
    monkeypatch.setattr(m, "_adapter_ws", {})
    got, go = [], threading.Barrier(4)

    def work():
        go.wait()
        got.append(m._adapter_workspace())

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4 and all(w is got[0] for w in got) and m._adapter_ws == {0: got[0]}
