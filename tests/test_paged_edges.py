"""Paged serving operators at their edges: calls in a row with nothing between
them, values and tables that the operators promise to leave alone, refusals."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_ref as ref
from test_paged import Batch, attn_case, check_attn, dev, params, run_attn, status_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_long_sgqa_gb300", "csrc")
gpu = pytest.mark.gpu
both = pytest.mark.parametrize("dtype", ["bf16", "fp32"])


@pytest.fixture(scope="module")
def s():
    from block_sparse_long_sgqa_gb300 import sgqa

    return sgqa


# ----------------------------------------------------------- calls in a row
def test_no_restrict_behind_a_dependent_launch():
    """A kernel that may start while the one before it still writes its inputs
    declares none of its pointers __restrict__."""
    seen = 0
    for name in os.listdir(CSRC):
        text = open(os.path.join(CSRC, name)).read()
        if not name.startswith("pa"):
            assert "launch_pdl" not in text, name
            continue
        for m in re.finditer(r"__global__[^{;]*", text):
            if "pdl_wait" in text[m.end():m.end() + 20000]:
                seen += 1
                assert "__restrict__" not in m.group(0), (name, m.group(0))
    assert seen >= 4


def test_no_way_past_the_wait_or_the_record():
    """Every way out of a kernel that others may depend on lies behind its wait, and
    the attention kernels' ways out leave the record that the merge reads."""
    seen = 0
    for name in os.listdir(CSRC):
        text = open(os.path.join(CSRC, name)).read()
        for part in re.split(r"pdl_next\(\);", text)[1:]:
            seen += 1
            assert not re.search(r"\breturn\b", part.split("pdl_wait();")[0]), name
    assert seen >= 6
    text = open(os.path.join(CSRC, "paged_attn_tc.cu")).read()
    early = re.search(r"& 1023u\) \{.*?return;", text, re.S).group(0)
    assert early.index("pdl_wait()") < early.index("a.rec[blockIdx.x] = make_int4(0, 0, 0, 0)")


@gpu
@both
def test_captured_chain_of_steps(s, dtype):
    """Several steps in one graph, each plan -> append -> attention -> release with
    nothing between the launches and the free counts in two buffers that take
    turns: every table, slot, count and output as in the step-by-step form."""
    rng = np.random.default_rng(21)
    g = torch.Generator().manual_seed(22)
    N, H, hk, d, ps, steps = 40, 4, 2, 64, 8, 5
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kv0 = rng.integers(0, 60, N)
    lens, cur = [], kv0
    for k in range(steps):
        q = np.where(rng.random(N) < 0.2, 0, rng.integers(0, 10, N))
        kv = cur + q
        cur = kv0 if k == steps - 1 else rng.integers(kv0, kv + 1)
        lens.append((q, kv, cur))  # the last release leaves the lengths of the start
    T = max(int(q.sum()) for q, _, _ in lens) + 3
    b = Batch(23, [0] * N, kv0, ps, spare=200, extra_cols=10, held_at="after")
    p = params(s, n_seqs=N, max_tokens=T, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=b.n_pages, max_pages=b.max_pages,
               dtype=s.BF16 if dtype == "bf16" else s.FP32)
    i32 = dict(dtype=torch.int32, device="cuda")
    free, table = dev(b.free), dev(b.table)
    nf, nf2 = torch.full((1,), b.n_free, **i32), torch.full((1,), -1, **i32)
    Kp, Vp = (torch.randn(b.n_pages, hk, ps, d, generator=g).to(dt) for _ in "kv")
    pool = [Kp.double().numpy(), Vp.double().numpy()]  # the host's copy
    Kp, Vp = Kp.cuda(), Vp.cuda()
    ws, st = s.alloc_paged_workspace(p), s.new_status()
    io = []
    for q, kv, keep in lens:
        x = torch.randn(T, H + 2 * hk, d, generator=g).to(dt)
        io.append(dict(
            q=dev(q).int(), kv=dev(kv).int(), keep=dev(keep).int(), host=x.double().numpy(),
            Q=x[:, :H].contiguous().cuda(), K=x[:, H:H + hk].contiguous().cuda(),
            V=x[:, H + hk:].contiguous().cuda(), q_start=torch.zeros(N + 1, **i32),
            slots=torch.zeros(T, dtype=torch.int64, device="cuda"), pos=torch.zeros(T, **i32),
            O=torch.zeros(T, H, d, dtype=dt, device="cuda"), lse=torch.zeros(H, T, device="cuda")))

    def chain():
        for v in io:
            s.sgqa_page_plan(p, v["q"], v["kv"], free, nf, table, v["q_start"], v["slots"],
                             v["pos"], nf2, status=st)
            s.sgqa_paged_append(p, v["K"], v["V"], v["slots"], Kp, Vp, status=st)
            s.sgqa_paged_attn(p, v["Q"], Kp, Vp, table, v["q_start"], v["kv"], v["O"], v["lse"],
                              ws, status=st)
            s.sgqa_page_release(p, v["kv"], v["keep"], table, free, nf2, nf, status=st)

    cg = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(cg):
        chain()
    h_table, h_free, h_n = b.table, b.free, b.n_free
    for it in range(4):  # three replays, then the same calls without a graph
        (cg.replay if it < 3 else chain)()
        assert status_of(s, st) == s.OK
        for v, (q, kv, keep) in zip(io, lens):
            h_table, q_start, slots, pos, h_n = ref.plan(q, kv, h_free, h_n, h_table, ps, T)
            assert np.array_equal(v["q_start"].cpu().numpy(), q_start)
            assert np.array_equal(v["slots"].cpu().numpy(), slots)
            assert np.array_equal(v["pos"].cpu().numpy(), pos)
            n = int(q_start[-1])
            for i, c0 in enumerate((H, H + hk)):
                pool[i][slots[:n] // ps, :, slots[:n] % ps] = v["host"][:n, c0:c0 + hk]
            R, z, tO, tl, mine = ref.attention(v["host"][:, :H], *pool, ps, h_table, q_start, kv,
                                               ref.default_scale(d), True, 0, dtype == "bf16")
            assert (np.abs(v["O"].double().cpu().numpy() - R)[mine] <= tO[mine]).all()
            assert (np.abs(v["lse"].double().cpu().numpy() - z)[:, mine] <= tl[:, mine]).all()
            h_free, h_n = ref.release(kv, keep, h_table, h_free, h_n, ps)
        assert nf.item() == h_n
        assert np.array_equal(free.cpu().numpy(), h_free)
        assert np.array_equal(table.cpu().numpy(), h_table)
        assert np.array_equal(Kp.double().cpu().numpy(), pool[0])
        assert np.array_equal(Vp.double().cpu().numpy(), pool[1])


# ------------------------------------------------------------ giving up a wait
def test_drains_do_not_hang_on_the_flag():
    """A role whose copies are all issued leaves before another role gives up, so
    it waits for them whether or not the flag is up by then."""
    text = open(os.path.join(CSRC, "paged_attn_tc.cu")).read()
    assert len(re.findall(r"mbar_wait_drain\(", text)) == 3 and "*up.flag != 0" not in text


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,kv", [([1], [100]), ([1, 1, 1], [250, 130, 7]), ([100], [150])])
def test_stalled_wait_of_a_short_request(s, monkeypatch, d, q, kv):
    """Requests of one or two key tiles, whose loads are all issued before the
    products' wait runs out: the status says so, the next call is right."""
    import test_paged

    monkeypatch.setitem(test_paged.ATTN, "stall", (q, kv, 8, 2, d, 16, {}))
    b, p, wide, K, V, q_start, kw = attn_case(s, "stall", "bf16")
    a = dict(Q=wide.cuda(), K_pages=K.cuda(), V_pages=V.cuda(), page_table=dev(b.table),
             q_start=dev(q_start), kv_len=dev(b.kv),
             O=torch.full(wide.shape, 3.0, dtype=wide.dtype, device="cuda"),
             lse=torch.full((p.n_q_heads, p.max_tokens), 7.0, device="cuda"),
             ws=s.alloc_paged_workspace(p))
    st = s.new_status()
    for _ in range(3):
        st[3] = s.DEBUG_STALL
        s.sgqa_paged_attn(p, **a, status=st)
        assert s.read_status(st) == (s.ERR_TIMEOUT, 220)
        s.reset_status(st)
        s.sgqa_paged_attn(p, **a, status=st)
        assert status_of(s, st) == s.OK
        check_attn(s, b, p, wide, K, V, q_start, kw, a["O"], a["lse"])


# ------------------------------------------------------------------- release
def run_release(s, b, kv, keep):
    p = params(s, n_seqs=b.N, max_tokens=0, page_size=b.ps, n_pages=b.n_pages,
               max_pages=b.max_pages)
    free, nf, st = dev(b.free), dev([b.n_free]).int(), s.new_status()
    out = torch.full_like(nf, 77)
    s.sgqa_page_release(p, dev(kv).int(), dev(keep).int(), dev(b.table), free, nf, out, status=st)
    return free.cpu().numpy(), out.item(), s.read_status(st)


def release_case(name):
    rng = np.random.default_rng(31)
    n, kv_max, ps = {"one": (1, 9, 8), "some": (60, 300, 16), "tiles": (4500, 60, 8),
                     "long": (40, 30000, 8), "one_long": (1, 600000, 8),
                     "most": (2100, 6000, 8)}[name]
    kv = rng.integers(1, kv_max, n)
    kv[0] = kv_max
    keep = np.where(rng.random(n) < 0.5, 0, rng.integers(0, kv + 1))
    keep[0] = min(keep[0], 17)
    return Batch(32, [0] * n, kv, ps, held_at="after"), kv, keep


RELEASES = ["one", "some", "tiles", "long", "one_long", "most"]


@gpu
@pytest.mark.parametrize("name", RELEASES)
def test_release_of_many_pages(s, name):
    """Pages that requests keep are not looked at, whatever their numbers."""
    b, kv, keep = release_case(name)
    for i in range(b.N):
        b.table[i, :ref.pages_of(int(keep[i]), b.ps)] = -1
    want, n_free = ref.release(kv, keep, b.table, b.free, b.n_free, b.ps)
    free, out, (code, _) = run_release(s, b, kv, keep)
    assert code == s.OK
    assert out == n_free and np.array_equal(free, want)


@gpu
@pytest.mark.parametrize("name", RELEASES)
def test_release_of_a_bad_page_gives_nothing_back(s, name):
    """A page number outside the pool among those given back refuses the call: the
    stack and its count stay."""
    b, kv, keep = release_case(name)
    back = [(i, c) for i in range(b.N)
            for c in range(ref.pages_of(int(keep[i]), b.ps), ref.pages_of(int(kv[i]), b.ps))]
    table = b.table.copy()
    for (i, c), bad in zip((back[0], back[-1], back[len(back) // 2], back[-len(back) // 3]),
                           (-1, b.n_pages, (1 << 31) - 1, -(1 << 31))):
        b.table = table.copy()
        b.table[i, c] = bad
        free, out, (code, detail) = run_release(s, b, kv, keep)
        assert (code, detail) == (s.ERR_BOUNDS, 314)
        assert out == b.n_free and np.array_equal(free[:out], b.free[:out])


# ------------------------------------------------------------ values at the edge
@gpu
@both
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", [100, 256, 700, 9000])
def test_nan_value_of_no_weight_is_seen(s, monkeypatch, dtype, d, kv):
    """A NaN among the values that a row sees makes that column of its output NaN,
    also where the weight, e^-200 of the row's, is 0 in 32 bits: in one tile, in
    tiles of both groups and in parts that are merged.  lse and the other columns
    are the ordinary ones."""
    import test_paged

    monkeypatch.setitem(test_paged.ATTN, "weightless", ([1, 1], [kv, 5], 8, 2, d, 16, {}))
    b, p, wide, K, V, q_start, kw = attn_case(s, "weightless", dtype)
    low = min(kv // 2, 128)  # keys before it have scores 200 below the others'
    wide[0, :, 0] = 16.0
    for j in range(kv):
        K[b.table[0, j // 16], :, j % 16, 0] = 0.0 if j < low else 200.0 * np.sqrt(d) / 16
    for j in (0, low // 2, low - 1):
        at = (int(b.table[0, j // 16]), 1, j % 16, 3)
        was = V[at].item()
        V[at] = float("nan")
        O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
        V[at] = was
        assert code == s.OK
        assert torch.isnan(O[0, 4:, 3]).all(), j
        O[0, 4:, 3] = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)[0][0, 4:, 3]
        check_attn(s, b, p, wide, K, V, q_start, kw, O, lse)


# ---------------------------------------------------------- a torch without CUDA
def test_host_entries_without_torch_cuda():
    """Sizing, planning and argument checks need no CUDA build of torch."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from block_sparse_long_sgqa_gb300 import sgqa as s
p = s.paged_params(3, 10, 8, 2, 64, 16, 20, 4)
assert s.paged_workspace_bytes(p) > 0
t = torch.zeros(20, dtype=torch.int32)
try:
    s.sgqa_page_release(p, t, t, t, t, t, t)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise SystemExit("a CPU tensor was taken")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
