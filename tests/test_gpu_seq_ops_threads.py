"""Handles of the sequence operators on host threads of one process: what one call
sets up is its own, or the same for all."""
import threading

import pytest
import torch

from recurrent_cell_unroll_gb300 import binding

pytestmark = pytest.mark.gpu


def test_short_backwards_of_two_threads():
    """Two handles, each on its thread and stream, with sequences of other lengths
    through the same kernel: no call refuses the other's."""
    lib, B, H, rounds = binding.load(), 310, 64, 4000
    codes, start = {}, threading.Barrier(2)

    def worker(T):
        ops, s = binding.SeqOps(), torch.cuda.Stream()
        with torch.cuda.stream(s):
            x = torch.randn(T, B, H, device="cuda").bfloat16()
            lam, st = torch.full((H,), -5.0, device="cuda"), torch.zeros(1, B, H, device="cuda")
            out = torch.empty_like(x)
            p, d = x.data_ptr(), out.data_ptr()
            args = (ops.h, binding.RCU_BF16, binding.RCU_BF16, 0, T, B, H, p, H, p, H, p, H, None, None,
                    None, lam.data_ptr(), 8.0, None, st.data_ptr(), p, H, None, d, H, None, 0, None, 0,
                    None, None, s.cuda_stream)
            start.wait()
            codes[T] = [lib.rcu_linrec_backward(*args) for _ in range(rounds)]
        s.synchronize()
        codes[T].append(ops.status(s))
        ops.close()

    threads = [threading.Thread(target=worker, args=(T,)) for T in (2, 20)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert set(codes) == {2, 20}
    for T, rc in codes.items():
        assert not any(rc), (T, sum(map(bool, rc)), "calls refused")
