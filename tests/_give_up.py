"""Child process of test_gpu_prefill_give_up.py: prefill calls in which chosen softmax warps give up their wait
for a piece's last product, then the same call again. One line per case: the flags and seconds of the
first, the flags of the second and its share of the error bound."""
import os
import sys
import time

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__)), os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]

import torch  # noqa: E402

import _bounds  # noqa: E402
import _operators as op  # noqa: E402
import paged_kv_cache_252_gb300 as pkv  # noqa: E402
from paged_kv_cache_252_gb300 import build  # noqa: E402
from test_gpu_prefill import Batch  # noqa: E402

CASES = [  # cache, new tokens, context lengths, softmax warps (bits 0..3 row tile 0, 4..7 row tile 1)
    ("fp16", [3], [20011], 0x01), ("fp16", [3], [20011], 0x06), ("fp16", [3], [20011], 0x0F),
    ("fp16", [300, 1], [9000, 700], 0x20), ("fp16", [300, 1], [9000, 700], 0xFF),
    ("int8", [3], [20011], 0x08), ("int8", [300, 1], [9000, 700], 0x41), ("bf16", [1100], [1100], 0x10)]


def main():
    dev = torch.device("cuda:0")
    pkv.load_library(build.build(variant="giveup"))
    for kv, ns, lens, warps in CASES:
        b = Batch(dev, kv, 128, 8, 2, ns, lens)
        b.status = torch.tensor([0, warps], dtype=torch.int32, device=dev)
        torch.cuda.synchronize()
        t = time.time()
        b.run()
        torch.cuda.synchronize()
        t = time.time() - t
        flags = b.status[0].item()
        b.status.zero_()
        b.out.fill_(7.5)
        b.run()
        torch.cuda.synchronize()
        share = max(op.assert_within(b.out[at], want, tol, "after") for at, want, tol in
                    (_bounds.attention_rows(b, s) for s in range(len(ns))))
        print(f"{kv} {ns} {warps:#x}: {flags} {t:.2f} {b.status[0].item()} {share:.2f}", flush=True)


if __name__ == "__main__":
    main()
