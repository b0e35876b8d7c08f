"""Host threads that call the router and the whole layer through one object: the launches of
a call must not mix with another call's that has the same workspace. On the CPU with a
library that only records, and on the GPU."""
import ctypes
import threading
import time

import pytest
import torch

import bit_quantized_moe_dequant_amd as mq


class Recorder:
    """In the library's place: every call takes a while, and notes calls that run at the same
    time over the same workspace."""

    def __init__(self):
        self.busy, self.mixed, self.seen, self.guard = set(), [], set(), threading.Lock()

    def _call(self, ws):
        with self.guard:
            self.seen.add(ws)
            if ws in self.busy:
                self.mixed.append(ws)
            self.busy.add(ws)
        time.sleep(0.002)
        with self.guard:
            self.busy.discard(ws)
        return 0

    def moeq_router_topk(self, r, x, T, ids, rw, ws, n, stream):
        return self._call(ws)

    def moeq_moe_forward(self, L, r, s, x, T, y, ids, rw, ws, n, stream):
        return self._call(ws)

    def moeq_router_workspace_bytes(self, r, T):
        return 256 * (T + 1)

    def moeq_moe_workspace_bytes(self, L, r, s, T):
        return 512 * (T + 1)

    def moeq_workspace_init(self, ws, n, stream):
        return 0


def in_threads(n, work):
    start, errors = threading.Barrier(n), []

    def body(i):
        try:
            start.wait()
            work(i)
        except Exception as e:  # reported by the caller
            errors.append(e)

    ts = [threading.Thread(target=body, args=(i,)) for i in range(n)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


def planes(fmt, rows, cols, n):
    return mq.Weight(fmt, rows, cols, n, torch.zeros(16, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8),
                     expert_stride=rows * cols, scale_expert_stride=rows * cols)


@pytest.mark.parametrize("given", [False, True])
def test_calls_do_not_mix_over_one_workspace(monkeypatch, given):
    lib = Recorder()
    monkeypatch.setattr(mq, "_LIB", lib)
    monkeypatch.setattr(mq, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(mq, "_stream_ptr", lambda: ctypes.c_void_p(0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    mq._gpu()
    monkeypatch.setattr(mq, "_GPU", (lambda: 0, lambda dev: 0) + mq._GPU[2:])
    router = mq.Router(torch.zeros((8, 64), dtype=torch.bfloat16), 2)
    layer = mq.Layer(64, 64, 8, 2, *(planes(mq.FMT_MXFP4, 64, 64, 8) for _ in range(3)))
    moe = mq.MoeLayer(layer, router)
    sizes = (1, 40, 3, 200)
    xs = [torch.zeros((T, 64), dtype=torch.bfloat16) for T in sizes]

    def work(i):
        for k in range(8):
            x = xs[(i + k) % len(xs)]
            mq.router_topk(router, x, ws=router.workspace(200) if given else None)
            mq.moe_forward(moe, x, ws=moe.workspace(200) if given else None)

    in_threads(4, work)
    assert lib.mixed == [] and lib.busy == set()
    if given:  # a workspace for more tokens serves fewer
        assert len(lib.seen) == 2


@pytest.mark.gpu
def test_threads_on_one_stream():
    """Two threads, one layer, the default stream: what each gets is what it gets alone."""
    from tests.test_gpu_moe import MX, Case, say
    say("threads")
    c = Case(512, 512, 12, 4, MX, MX, 256, seed=120)
    sizes = [(1, 8, 20, 100, 200), (3, 16, 70, 2, 130)]
    xs = [[c.x(T, 700 + 10 * i + j)[1] for j, T in enumerate(ts)] for i, ts in enumerate(sizes)]
    alone = [[mq.moe_forward(c.moe, x) + mq.router_topk(c.router, x) for x in v] for v in xs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        torch.cuda.set_device(0)
        for _ in range(20):
            for j, x in enumerate(xs[i]):
                got[i].append((j, mq.moe_forward(c.moe, x) + mq.router_topk(c.router, x)))

    in_threads(2, work)
    torch.cuda.synchronize()
    for i in range(2):
        for j, out in got[i]:
            for a, b in zip(out, alone[i][j]):
                assert torch.equal(a, b), (i, j)
