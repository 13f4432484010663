"""The serving operators called from several host threads at once: on streams of their own, and all on one."""
import threading

import pytest
import torch

import _operators as op
from test_gpu_prefill import Batch, dev  # noqa: F401

pytestmark = pytest.mark.gpu


class Job:
    """A thread's calls: rotary write, prefill over workspaces that grow, acceptance; outputs of every turn."""

    SHAPES = [([40], [300]), ([300, 1], [6000, 900]), ([3], [20011])]

    def __init__(self, dev, kv, seed):
        import paged_kv_cache_252_gb300 as pkv
        self.pkv = pkv
        self.batches = [Batch(dev, kv, 128, 8, 2, ns, lens, seed=seed + i) for i, (ns, lens) in enumerate(self.SHAPES)]
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        T = 64
        self.kc, self.vc, self.sc = op.make_cache(kv, 8, 2, 128, g, dev)
        self.x = [torch.randn((T, h, 128), generator=g, device=dev).to(op.src_dtype(kv)) for h in (8, 2, 2)]
        self.q = torch.empty_like(self.x[0])
        self.pos = torch.arange(seed, seed + T, device=dev)
        self.slots = torch.randperm(128, generator=g, device=dev)[:T].to(torch.int32)
        self.inv, _ = pkv.rotary_inv_freq(128, device=dev)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
        self.accept = (i32([[0, 1, 2, 3, 4, 5, 6, 7]]), i32([100]), i32([[3, 5, 9, 9]]), i32([4]), i32([0]))

    def turn(self):
        for b in self.batches:
            b.run()
        self.pkv.rotary_write(self.q, *self.x, self.pos, self.slots, self.kc, self.vc, self.inv, scales=self.sc)
        bt, cl, acc, num, new = self.accept
        self.pkv.kv_cache_accept(self.kc, self.vc, bt, cl, acc, num, new, 20, scales=self.sc)

    def state(self):
        return [b.out.clone() for b in self.batches] + [t.clone() for t in (self.q, self.kc, self.vc, self.accept[-1])]


@pytest.mark.parametrize("own_streams", [True, False], ids=["streams", "one-stream"])
def test_threads_do_not_disturb_one_another(dev, own_streams):  # noqa: F811
    kvs = ["bf16", "int8", "e5m2", "fp16"]
    jobs, alone = ([Job(dev, kv, 10 * i) for i, kv in enumerate(kvs)] for _ in range(2))
    for j in alone:
        for _ in range(20):
            j.turn()
    torch.cuda.synchronize()
    errors, gate = [], threading.Barrier(len(jobs))

    def work(job):
        try:
            stream = torch.cuda.Stream() if own_streams else torch.cuda.default_stream()
            gate.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(20):
                    job.turn()
            stream.synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for got, want in zip(jobs, alone):
        for a, b in zip(got.state(), want.state()):
            assert torch.equal(a, b)
        assert all(b.status.item() == 0 for b in got.batches)
