"""Calls from several host threads, each on its own stream and buffers."""
import threading

import pytest
import torch

gpu = pytest.mark.gpu


@gpu
def test_unions_of_two_host_threads():
    """Caches of very different lengths selected from at once: the shared memory that one call
    asks for does not depend on the other's, and neither do the results."""
    from block_sparse_long_sgqa_gb300 import sgqa as s

    fail, same, gate = [], [], threading.Barrier(2)

    def work(kv):
        with torch.cuda.stream(torch.cuda.Stream()):
            p = s.params(seq_q=64, seq_kv=kv, q_offset=kv - 64, n_q_heads=1, n_kv_heads=1, head_dim=64,
                         block_size=8, topk_tokens=4096, tile_q=64)
            scores = torch.randn(1, 64, kv // 8, device="cuda")
            sel = torch.zeros(1, 64, 512, dtype=torch.int32, device="cuda")
            u, st, first = s.alloc_union(p), s.new_status(), None
            gate.wait()
            try:
                for _ in range(1500):
                    s.sgqa_topk_union(p, scores, 0, 64, sel, *u, status=st)
                    if first is None:
                        first = [x.clone() for x in (sel, u[0], u[1], u[2], u[3])]
                assert s.read_status(st)[0] == s.OK
                same.append(all(torch.equal(a, b) for a, b in zip(first, (sel, *u))))
            except Exception as e:
                fail.append(e)
    threads = [threading.Thread(target=work, args=(kv,)) for kv in (8192, 1 << 20)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fail, fail
    assert same == [True, True]
