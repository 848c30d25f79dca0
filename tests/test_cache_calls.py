"""Calls of the operators around the paged cache that their documentation allows or
refuses: outputs on inputs, host threads at once, forms that the ordinary sizes do not reach."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import paged_ref as ref
from test_cache_ops import (PLANS, VALUES, VERIFIES, MassCase, VerifyCase, check_plan, dev,
                            plan_case)
from test_paged import params, status_of

gpu = pytest.mark.gpu
# Addresses that nothing may read: where a refusal were missing, the call would.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls with made-up addresses")


@pytest.fixture(scope="module")
def s():
    from block_sparse_long_sgqa_gb300 import sgqa

    return sgqa


def clashes(inputs, outputs, allowed=()):
    """(output, address) for each output placed on each other buffer: at its start, and so
    that its last or first word is the other's first or last."""
    sizes = {**inputs, **outputs}
    base = {k: (i + 1) << 32 for i, k in enumerate(sizes)}
    for o in outputs:
        for b in sizes:
            if b == o:
                continue
            places = [base[b] - outputs[o] + 4, base[b] + sizes[b] - 4]
            if (o, b) not in allowed:
                places.append(base[b])
            for x in places:
                yield o, b, {**base, o: x}


# -------------------------------------------------------------- verification
@no_gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_verify_refuses_outputs_on_inputs(s, dtype):
    n, t, v, e = 5, 17, 100, 4 if dtype == "fp32" else 2
    p = s.verify_params(n, t, v, s.FP32 if e == 4 else s.BF16, p_stride=104, d_stride=112)
    inputs = dict(P=((t - 1) * 104 + v) * e, D=((t - 1) * 112 + v) * e, tokens=4 * t, q_start=4 * n + 4,
                  kv_len=4 * n, u=4 * t, u_next=4 * n)
    outputs = dict(n_accepted=4 * n, next_token=4 * n, keep_len=4 * n)
    for o, b, at in clashes(inputs, outputs, allowed=[("keep_len", "kv_len")]):
        rc = s._lib.sgqa_draft_verify(ctypes.byref(p), *at.values(), None, None)
        assert rc == s.ERR_INVALID_ARG, (o, b)


@gpu
@pytest.mark.parametrize("name", VERIFIES)
def test_verify_lengths_in_place(s, name):
    """keep_len on kv_len, from caches no longer than the drafts (so that the new length would
    not hold them): as with a buffer of its own."""
    c = VerifyCase(s, name)
    c.kv = np.diff(c.q_start).astype(np.int32)
    for _ in range(10):
        kv = dev(c.kv).clone()
        c.out["keep_len"] = kv
        assert c.run(s, kv_len=kv) == s.OK
        c.check()


@gpu
def test_verify_lengths_in_place_many(s, monkeypatch):
    """The same with more requests than fit the SMs at a time."""
    monkeypatch.setitem(VERIFIES, "crowd", ([2] * 400, 20000, True, "bf16", 0))
    c = VerifyCase(s, "crowd")
    c.kv = np.diff(c.q_start).astype(np.int32)
    for _ in range(5):
        kv = dev(c.kv).clone()
        c.out["keep_len"] = kv
        assert c.run(s, kv_len=kv) == s.OK
        c.check()


# ------------------------------------------------------------------ eviction
@no_gpu
@pytest.mark.parametrize("optional", [True, False])
def test_plan_refuses_outputs_on_inputs(s, optional):
    """(kv_len_out on next_pos, say, would change what other groups of the request take for
    recent.)"""
    n, hk, ps, pages, cols, budget = 3, 2, 16, 20, 4, 6
    p = params(s, n_seqs=n, n_kv_heads=hk, page_size=ps, n_pages=pages, max_pages=cols)
    inputs = dict(mass_pages=4 * pages * hk * ps, pos_pages=4 * pages * hk * ps, page_table=4 * n * cols,
                  kv_len=4 * n, next_pos=4 * n)
    outputs = dict(n_moves=4 * n * hk, moves=8 * n * hk * budget, kv_len_out=4 * n)
    for o, b, at in clashes(inputs, outputs):
        if not optional:
            at.update(pos_pages=None, next_pos=None)
            if b in ("pos_pages", "next_pos"):
                continue
        rc = s._lib.sgqa_evict_plan(ctypes.byref(p), budget, 1, 1, *at.values(), None, None)
        assert rc == s.ERR_INVALID_ARG, (o, b)


CLUSTERS = {  # blocks of a (request, group) by the table's places and by how many there are of them
    "four_idle": ([20000, 30, 16400], 2, 64, 3000, 50, 4, 0),           # 20032 places, 6 of them
    "two_full": ([32800, 5000] + [40] * 36, 4, 32, 4096, 7, 3, 0),      # 32800 places, 152
    "four_full": ([66000, 300] + [40] * 36, 4, 32, 10000, 0, 0, 0),     # 66016 places, 152
    "eight_full": ([140000, 9] + [40] * 36, 4, 64, 20000, 100, 9, 0),   # 140032 places, 152
}


@gpu
@pytest.mark.parametrize("with_pos", [True, False])
@pytest.mark.parametrize("values", VALUES)
@pytest.mark.parametrize("name", CLUSTERS)
def test_plan_clusters(s, name, values, with_pos, monkeypatch):
    monkeypatch.setitem(PLANS, name, CLUSTERS[name])
    _, p, t, want = plan_case(s, name, values, with_pos=with_pos)
    st = s.new_status()
    s.sgqa_evict_plan(p, **t, status=st)
    assert status_of(s, st) == s.OK
    check_plan(t, want)


@gpu
def test_plans_of_two_host_threads(s):
    """Tables of different widths, planned from two threads at once: the shared memory that one
    call asks for does not depend on the other's."""
    n, hk, ps, kv, budget, rounds = 38, 4, 64, 100, 60, 3000  # a block a (request, group)
    fail, got, gate = [], [None, None], threading.Barrier(2)

    def work(i, max_pages):
        p = params(s, n_seqs=n, max_tokens=0, n_q_heads=hk, n_kv_heads=hk, page_size=ps, n_pages=2,
                   max_pages=max_pages)
        i32 = dict(dtype=torch.int32, device="cuda")
        with torch.cuda.stream(torch.cuda.Stream()):
            mass = torch.arange(2 * hk * ps, dtype=torch.float32, device="cuda")
            table = torch.zeros(n, max_pages, **i32)
            table[:, 1] = 1
            lens = torch.full((n,), kv, **i32)
            out = [torch.zeros(n, hk, **i32), torch.zeros(n, hk, budget, 2, **i32), torch.zeros(n, **i32)]
            status = s.new_status()
            gate.wait()
            try:
                for _ in range(rounds):
                    s.sgqa_evict_plan(p, mass, table, lens, *out, budget=budget, status=status)
                assert status_of(s, status) == s.OK
                got[i] = [x.cpu() for x in out]
            except Exception as e:
                fail.append(e)
    # 12800 and 32768 keys a block: 50 and 128 KB
    threads = [threading.Thread(target=work, args=a) for a in ((0, 200), (1, 512))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fail, fail
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0] == kv - budget).all()


@gpu
def test_move_counts_above_the_table(s):
    """More moves than the table has places cannot be distinct: none is carried out, even
    where the budget would allow them."""
    ps, cols, budget = 8, 4, 100
    p = params(s, n_seqs=2, max_tokens=0, n_q_heads=1, n_kv_heads=1, page_size=ps, n_pages=8, max_pages=cols)
    K = torch.randn(8, 1, ps, 64).to(torch.bfloat16).cuda()
    V = K.flip(0).contiguous()
    table = torch.arange(8, dtype=torch.int32).view(2, cols).cuda()
    moves = torch.zeros(2, 1, budget, 2, dtype=torch.int32)
    moves[:, 0, :, 0], moves[:, 0, :, 1] = 31, torch.arange(budget)
    counts = torch.tensor([[33], [1]], dtype=torch.int32)
    k, v, st = K.clone(), V.clone(), s.new_status()
    s.sgqa_evict_move(p, table, counts.cuda(), moves.cuda(), k, v, budget, status=st)
    assert s.read_status(st) == (s.ERR_BOUNDS, 381)
    for x, y in ((k, K), (v, V)):
        y[4, 0, 0] = y[7, 0, 7]  # the second request's one move
        assert torch.equal(x, y)


# ------------------------------------------------------- accumulated weights
def entries_of(c, i, j):
    """Mask of the entries of cached positions j of request i, in every group."""
    m = np.zeros(c.old.shape, bool)
    m[c.b.table[i, j // c.ps], :, j % c.ps] = True
    return m


@no_gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("with_pos", [True, False])
def test_mass_refuses_outputs_on_inputs(s, dtype, with_pos):
    n, t, h, hk, d, ps, pages, cols, e = 3, 11, 8, 2, 64, 16, 20, 4, 2 if dtype == "bf16" else 4
    p = params(s, n_seqs=n, max_tokens=t, n_q_heads=h, n_kv_heads=hk, page_size=ps, n_pages=pages,
               max_pages=cols, dtype=s.BF16 if e == 2 else s.FP32, q_stride=(h + 4) * d)
    need = s.mass_workspace_bytes(p)
    entries = pages * hk * ps
    inputs = dict(Q=((t - 1) * (h + 4) + h) * d * e, K_pages=entries * d * e, page_table=4 * n * cols,
                  q_start=4 * n + 4, kv_len=4 * n, lse=4 * h * t, mass_in=4 * entries, positions=4 * t)
    outputs = dict(mass_out=4 * entries, pos_pages=4 * entries, ws=need)
    order = ("Q", "K_pages", "page_table", "q_start", "kv_len", "lse", "mass_in", "mass_out", "positions",
             "pos_pages", "ws")
    for o, b, at in clashes(inputs, outputs, allowed=[("mass_out", "mass_in")]):
        if not with_pos:
            if "pos_pages" in (o, b) or b == "positions":
                continue
            at.update(positions=None, pos_pages=None)
        a = [at[k] for k in order]
        rc = s._lib.sgqa_paged_mass(ctypes.byref(p), *a[:6], 0, *a[6:], need, None, None)
        assert rc == s.ERR_INVALID_ARG, (o, b)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["decode", "chunks", "heads", "window", "full", "observe", "many", "cut",
                                  "mix", "mix_window", "mix_full", "mix_ends", "wide"])
def test_mass_leaves_out_marked_rows(s, name, value, dtype):
    """Rows whose lse is -infinity add nothing, whatever they hold, and neither do keys that only
    such rows see."""
    c = MassCase(s, name, dtype, seed=3)
    rng = np.random.default_rng(4)
    out = rng.random(c.lse.shape) < 0.2
    Q, K = c.t["Q"], c.t["K_pages"]
    for i, (a, n) in enumerate(zip(c.q, c.kv)):
        if c.causal and 1 < a <= n:  # the last token, and with it the last key
            out[:, c.q_start[i + 1] - 1] = True
            K[int(c.b.table[i, (n - 1) // c.ps]), :, (n - 1) % c.ps] = value
    c.lse[out] = -np.inf
    c.t["lse"].copy_(torch.tensor(c.lse))
    Q[torch.tensor(out.T.copy()).cuda()] = value
    for _ in range(3):
        assert c.run(s) == s.OK
        c.check()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", ["decode", "cut", "mix", "mix_full", "mix_ends_few", "many"])
def test_marked_rows_change_no_other_request(s, name, dtype):
    """One row marked in one request: the others' entries keep their bits, and a repeated call
    repeats all."""
    c = MassCase(s, name, dtype)
    assert c.run(s) == s.OK
    before = c.t["mass_out"].clone()
    c.t["lse"][0, int(c.q_start[1]) - 1] = -float("inf")
    first = None
    for _ in range(10):
        c.t["mass_out"].fill_(77.0)
        assert c.run(s) == s.OK
        got = c.t["mass_out"].clone()
        first = got if first is None else first
        assert torch.equal(got.view(torch.int32), first.view(torch.int32))
    mine = torch.tensor(entries_of(c, 0, np.arange(c.kv[0]))).cuda()
    assert torch.equal(got[~mine].view(torch.int32), before[~mine].view(torch.int32))
    assert not torch.equal(got[mine], before[mine])


@gpu
@pytest.mark.parametrize("dtype,scale", [("bf16", 2.0 ** -64), ("bf16", 1e-6), ("bf16", 0.02), ("bf16", 1.0),
                                         ("bf16", 3.0), ("fp32", 1e-30), ("fp32", 2.0 ** -64), ("fp32", 0.02),
                                         ("fp32", 1.0), ("fp32", 3.0)])
@pytest.mark.parametrize("name", ["decode", "chunks", "cut", "window"])
def test_mass_other_scales(s, name, dtype, scale):
    """Scales from one under which all keys weigh the same to one under which one key has it all."""
    c = MassCase(s, name, dtype, seed=6)
    c.scale = float(np.float32(scale))
    _, lse, _, _, _ = ref.attention(c.Q64, c.K64, np.zeros_like(c.K64), c.ps, c.b.table, c.q_start, c.kv,
                                    c.scale, c.causal, c.window, dtype == "bf16")
    c.lse = lse.astype(np.float32)
    c.t["lse"].copy_(torch.tensor(c.lse))
    c.p.softmax_scale = scale
    assert c.run(s) == s.OK
    c.check()
