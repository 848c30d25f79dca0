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


def request_hit(p, q_start, i, g=None):
    """[T][H] mask of request i's rows (of KV head g's heads)."""
    G = p.n_q_heads // p.n_kv_heads
    hit = torch.zeros(p.max_tokens, p.n_q_heads, dtype=torch.bool, device="cuda")
    hit[q_start[i]:q_start[i + 1], slice(None) if g is None else slice(g * G, (g + 1) * G)] = True
    return hit


EDGE = ["decode", "decode_long", "few_g16", "chunk", "mixed_idle"]


@gpu
@both
@pytest.mark.parametrize("name", EDGE)
def test_scores_of_minus_infinity(s, name, dtype):
    """Keys whose scores are -infinity have no weight; a row all of whose scores
    are is one that sees nothing.  Other requests keep their bits."""
    b, p, wide, K, V, q_start, kw = attn_case(s, name, dtype)
    i = int(np.argmax(b.kv * (b.q > 0)))
    rows = slice(int(q_start[i]), int(q_start[i + 1]))
    wide[rows, :, 5] = wide[rows, :, 5].abs() + 0.5
    first = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    n, hit = int(b.kv[i]), request_hit(p, q_start, i)
    half = max(1, int(n - b.q[i]) // 2)
    for upto in (half, n):
        K2, K64 = K.clone(), K.clone()
        for j in range(upto):
            K2[b.table[i, j // b.ps], :, j % b.ps, 5] = -float("inf")
            K64[b.table[i, j // b.ps], :, j % b.ps, 5] = -4096.0  # a weight below e^-100
        O, lse, code = run_attn(s, p, wide, K2, V, b.table, q_start, b.kv)
        assert code == s.OK
        assert torch.equal(O[~hit], first[0][~hit]) and torch.equal(lse.T[~hit], first[1].T[~hit])
        if upto == n:
            assert (O[hit] == 0).all() and torch.isneginf(lse.T[hit]).all()
        else:
            check_attn(s, b, p, wide, K64, V, q_start, kw, O, lse)


@gpu
@both
@pytest.mark.parametrize("name", ["decode", "decode_long", "few_g16", "decode_split_16"])
def test_infinite_scores_and_values(s, name, dtype):
    """A score of +infinity makes a row's O and lse NaN; an infinite value makes its
    column of O infinite and leaves lse and the other columns.  Single tokens."""
    b, p, wide, K, V, q_start, kw = attn_case(s, name, dtype)
    i, g = int(np.argmax(b.kv * (b.q > 0))), p.n_kv_heads - 1
    t, hit = int(q_start[i]), request_hit(p, q_start, i, g)
    wide[t, :, 5] = wide[t, :, 5].abs() + 0.5
    O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    for j in (0, int(b.kv[i]) // 2, int(b.kv[i]) - 1):
        at = (int(b.table[i, j // b.ps]), g, j % b.ps, 5)
        K2, V2 = K.clone(), V.clone()
        K2[at] = float("inf")
        Oi, li, code = run_attn(s, p, wide, K2, V, b.table, q_start, b.kv)
        assert code == s.OK
        assert torch.isnan(Oi[hit]).all() and torch.isnan(li.T[hit]).all()
        assert torch.equal(Oi[~hit], O[~hit]) and torch.equal(li.T[~hit], lse.T[~hit])
        V2[at] = -float("inf")
        Oi, li, code = run_attn(s, p, wide, K, V2, b.table, q_start, b.kv)
        assert code == s.OK
        assert torch.isneginf(Oi[hit][:, 5]).all()
        Oi[..., 5][hit] = O[..., 5][hit]
        assert torch.equal(Oi, O) and torch.equal(li, lse)


# --------------------------------------------- what lies before a window, bad pages
WINDOWS = {
    # single tokens and drafts whose windows begin at every offset of a page
    "one": ([1] * 40, [300 + i for i in range(40)], 16, 2, 128, 24, dict(window=100)),
    "one_d64": ([1] * 40, [250 + i for i in range(40)], 32, 2, 64, 32, dict(window=130)),
    "drafts": ([5] * 20, [700 + i for i in range(20)], 16, 2, 128, 16, dict(window=65)),
    "chunks": ([150, 80, 1, 33], [900, 505, 400, 290], 16, 4, 128, 40, dict(window=77)),
    "chunks_d64": ([300, 41], [1000, 600], 8, 1, 64, 64, dict(window=200)),
    "long": ([1, 1], [30000, 20001], 8, 1, 128, 64, dict(window=9000)),
    "first": ([1, 20], [600, 700], 8, 2, 64, 8, dict(window=1)),
}


@gpu
@both
@pytest.mark.parametrize("name", WINDOWS)
def test_what_lies_before_a_window_has_no_effect(s, monkeypatch, name, dtype):
    """Keys and values before the first position that a request's rows see hold NaN
    and infinities, and the pages that lie wholly before it have no valid number."""
    import test_paged

    monkeypatch.setitem(test_paged.ATTN, "before", WINDOWS[name])
    b, p, wide, K, V, q_start, kw = attn_case(s, "before", dtype)
    bad = [-1, b.n_pages, -(1 << 31), (1 << 31) - 1]
    for i in range(b.N):
        lo = max(0, int(b.kv[i] - b.q[i]) + 1 - p.window)
        for j in range(lo):
            K[b.table[i, j // b.ps], :, j % b.ps] = float("nan") if j % 3 else float("inf")
            V[b.table[i, j // b.ps], :, j % b.ps] = float("nan") if j % 2 else -float("inf")
        b.table[i, :lo // b.ps] = [bad[c % 4] for c in range(lo // b.ps)]
    O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    assert code == s.OK
    check_attn(s, b, p, wide, K, V, q_start, kw, O, lse)


@gpu
@both
@pytest.mark.parametrize("d", [64, 128])
def test_what_other_items_see_has_no_effect(s, monkeypatch, dtype, d):
    """A NaN that only the first rows of a windowed chunk see stays within 256 (token,
    head) rows of them."""
    import test_paged

    monkeypatch.setitem(test_paged.ATTN, "items", ([400], [900], 8, 2, d, 16, dict(window=90)))
    b, p, wide, K, V, q_start, kw = attn_case(s, "items", dtype)
    O, lse, _ = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    j = 500 + 1 - 90  # the first position that token 0 (at 500) sees, and only it
    K[b.table[0, j // 16], :, j % 16] = float("nan")
    V[b.table[0, j // 16], :, j % 16] = float("nan")
    On, ln, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    assert code == s.OK
    assert torch.isnan(On[0]).all() and torch.isnan(ln[:, 0]).all()
    assert torch.equal(On[64:], O[64:]) and torch.equal(ln[:, 64:], lse[:, 64:])
    assert torch.equal(ln[:, 1:], lse[:, 1:])  # scores that a row does not see are left out


@gpu
@both
@pytest.mark.parametrize("name", ["decode_long", "chunk", "mixed_idle", "few_two_tokens", "window"])
def test_bad_pages_read_as_zeros(s, name, dtype):
    b, p, wide, K, V, q_start, kw = attn_case(s, name, dtype)
    i = int(np.argmax(b.kv * (b.q > 0)))
    c = ref.pages_of(int(b.kv[i]), b.ps) - 2
    zero = torch.zeros_like(K[:1])
    K64, V64, good = torch.cat([K, zero]), torch.cat([V, zero]), b.table.copy()
    for bad in (-1, b.n_pages, -(1 << 31), (1 << 31) - 1):
        b.table = good.copy()
        b.table[i, c] = bad
        O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
        assert code == s.ERR_BOUNDS
        b.table[i, c] = b.n_pages  # the zero page of the 64-bit form
        check_attn(s, b, p, wide, K64, V64, q_start, kw, O, lse)


# ------------------------------------------------------------------- large ones
@gpu
@both
def test_waves_among_other_requests(s, dtype):
    """Requests that go out in waves beside single tokens, an idle one and a short
    prompt; checked on spread rows."""
    d, hk, ps = 128, 8, 64
    H = 64 if dtype == "bf16" else 16
    b = Batch(8, [1, 700, 0, 650, 30, 1], [3000, 20011, 50, 15000, 30, 9000], ps, held_at="after")
    q_start = np.concatenate([[0], np.cumsum(b.q)]).astype(np.int32)
    T = int(q_start[-1]) + 5
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    p = params(s, n_seqs=b.N, max_tokens=T, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=b.n_pages, max_pages=b.max_pages,
               dtype=s.BF16 if dtype == "bf16" else s.FP32)
    torch.manual_seed(3)
    Q = torch.randn(T, H, d, device="cuda").to(dt)
    K, V = (torch.randn(b.n_pages, hk, ps, d, device="cuda").to(dt) for _ in "KV")
    O, lse, code = run_attn(s, p, Q.cpu(), K, V, b.table, q_start, b.kv)
    assert code == s.OK
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (O[-5:] == 3.0).all() and (lse[:, -5:] == 7.0).all()
    assert np.isfinite(O).all() and np.isfinite(lse).all()
    Kn, Vn, Qn = (x.double().cpu().numpy() for x in (K, V, Q))
    for r in range(b.N):
        for i in sorted({0, 1, 31, 32, 333, int(b.q[r]) - 1}):
            if not 0 <= i < int(b.q[r]):
                continue
            t, n = int(q_start[r]) + i, int(b.kv[r] - b.q[r]) + i + 1
            R, z, tO, tl, _ = ref.attention(Qn[t:t + 1], Kn, Vn, ps, b.table[r:r + 1], [0, 1], [n],
                                            ref.default_scale(d), True, 0, dtype == "bf16")
            assert (np.abs(O[t] - R[0]) <= tO[0]).all(), (r, i)
            assert (np.abs(lse[:, t] - z[:, 0]) <= tl[:, 0]).all(), (r, i)


@gpu
@pytest.mark.parametrize("T", [1, 150])
def test_fp32_offsets_past_4_gib(s, T):
    """fp32 pages at the far end of a pool of more than 4 GiB, by the kernel for few
    rows and the one for many."""
    d, hk, H, ps, n_pages = 128, 8, 16, 64, 20000  # 5.2 GB for K, as much for V
    p = params(s, n_seqs=1, max_tokens=T, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=n_pages, max_pages=3, dtype=s.FP32)
    Kp, Vp = (torch.zeros(n_pages, hk, ps, d, device="cuda") for _ in "KV")
    torch.manual_seed(4)
    K, V = (torch.randn(150, hk, d, device="cuda") for _ in "KV")
    Q = torch.randn(T, H, d, device="cuda")
    table = np.array([[n_pages - 1, 2, n_pages - 2]], np.int32)
    pos = np.arange(150)
    slots = table[0, pos // ps].astype(np.int64) * ps + pos % ps
    st = s.new_status()
    pa = params(s, n_seqs=1, max_tokens=150, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
                n_pages=n_pages, max_pages=3, dtype=s.FP32)
    s.sgqa_paged_append(pa, K, V, dev(slots), Kp, Vp, status=st)
    O, lse = torch.zeros_like(Q), torch.zeros(H, T, device="cuda")
    s.sgqa_paged_attn(p, Q, Kp, Vp, dev(table), dev(np.array([0, T], np.int32)),
                      dev(np.array([150], np.int32)), O, lse, s.alloc_paged_workspace(p), status=st)
    assert status_of(s, st) == s.OK
    assert torch.equal(Kp[n_pages - 1].transpose(0, 1), K[:64])
    used = Kp.flatten(1).any(1).nonzero().flatten().tolist()
    assert used == [2, n_pages - 2, n_pages - 1]
    Kl, Vl = (x.double().cpu().numpy().transpose(1, 0, 2)[None] for x in (K, V))
    R, z, tO, tl, _ = ref.attention(Q.double().cpu().numpy(), Kl, Vl, 150, np.zeros((1, 1), int),
                                    [0, T], [150], ref.default_scale(d), True, 0, False)
    assert (np.abs(O.double().cpu().numpy() - R) <= tO).all()
    assert (np.abs(lse.double().cpu().numpy() - z) <= tl).all()


# ------------------------------------------- the sparse layer on the same pages
@gpu
def test_sparse_layer_on_planned_pages(s):
    """A ragged batch through both kinds of layer over pools and tables that the
    plan and the append made: the sparse layer takes a request at a time, on its row
    of the page table, with the request's length as seq_kv.  Prompts, then a
    decode step, against the oracle; the dense layer's decode step beside it."""
    import oracle
    from block_sparse_long_sgqa_gb300 import synth
    from helpers import clear_margin, r3_check

    ps, lens = 16, [700, 333, 41]
    wls = [synth.WORKLOADS["gqa_32k"].replace(name="planned", seq_q=n + 1, seq_kv=n + 1,
                                              topk_tokens=128, seed=77 + n) for n in lens]
    inp = [synth.make_inputs(w) for w in wls]
    rows = lambda x: torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).cuda().view(torch.bfloat16)
    H, hk, d = wls[0].n_q_heads, wls[0].n_kv_heads, wls[0].head_dim
    N, n_pages, max_pages, T = len(lens), 90, 60, sum(lens) + 9
    i32 = dict(dtype=torch.int32, device="cuda")
    free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).int().cuda()
    nf, nf2 = torch.full((1,), n_pages, **i32), torch.zeros(1, **i32)
    table, st = torch.full((N, max_pages), -1, **i32), s.new_status()
    Kp, Vp = (torch.full((n_pages, hk, ps, d), float("nan"), device="cuda").bfloat16() for _ in "kv")

    def step(q, kv, T, parts):
        """Plans and appends one step; parts(name): the rows of all requests."""
        pp = params(s, n_seqs=N, max_tokens=T, n_q_heads=H, n_kv_heads=hk, head_dim=d,
                    page_size=ps, n_pages=n_pages, max_pages=max_pages)
        q_start, pos = torch.zeros(N + 1, **i32), torch.zeros(T, **i32)
        slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        s.sgqa_page_plan(pp, dev(q).int(), dev(kv).int(), free, nf, table, q_start, slots, pos, nf2,
                         status=st)
        nf.copy_(nf2)
        pad = T - sum(q)
        x = {k: torch.cat([parts(k), torch.zeros(pad, (H if k == "Q" else hk), d, device="cuda",
                                                 dtype=torch.bfloat16)]) for k in "QKV"}
        s.sgqa_paged_append(pp, x["K"], x["V"], slots, Kp, Vp, status=st)
        return pp, q_start, x["Q"]

    def check(O, lse, i, r, q_offset):
        w = wls[i].replace(seq_q=len(r), q_offset=q_offset)
        Qf, Kf, Vf = (synth.widen(inp[i][k]) for k in "QKV")
        n = q_offset + len(r)
        w = w.replace(seq_kv=n)
        S, _, O64, l64 = oracle.prefill_rows(Qf[q_offset:n], Kf[:n], Vf[:n], q_offset, w.block_size,
                                             w.k_blocks, r)
        mask = np.repeat(clear_margin(S, w, r).T, H // hk, axis=1)
        assert mask.mean() >= 0.5
        r3_check(O.float().cpu().numpy(), lse.cpu().numpy(), O64, l64, mask)

    # the prompts
    step(lens, lens, T, lambda k: torch.cat([rows(x[k][:n]) for x, n in zip(inp, lens)]))
    for i, n in enumerate(lens):
        p = s.params_for(wls[i].replace(seq_q=n, seq_kv=n, page_size=ps))
        O, lse = s.alloc_outputs(p)
        s.sgqa_prefill(p, rows(inp[i]["Q"][:n]), Kp, Vp, s.kbar_empty(p), O, lse,
                       s.alloc_workspace(p, s.WS_PREFILL), page_table=table[i], status=st)
        assert status_of(s, st) == s.OK
        check(O, lse, i, np.arange(n, dtype=np.int32), 0)
    # a decode step of all of them
    after = [n + 1 for n in lens]
    pp, q_start, Q = step([1] * N, after, N + 2, lambda k: torch.cat(
        [rows(x[k][n:n + 1]) for x, n in zip(inp, lens)]))
    for i, n in enumerate(lens):
        p = s.params_for(wls[i].replace(seq_q=1, q_offset=n, page_size=ps))
        O, lse = s.alloc_outputs(p)
        cache = s.KeyCache(p, cap_blocks=(n + 1) // wls[i].block_size + 64)
        s.sgqa_decode(p, Q[i:i + 1].contiguous(), Kp, Vp, cache, O, lse,
                      s.alloc_workspace(p, s.WS_DECODE), page_table=table[i], status=st)
        assert status_of(s, st) == s.OK
        check(O, lse, i, np.arange(1, dtype=np.int32), n)
    O, lse = torch.zeros_like(Q), torch.zeros(H, N + 2, device="cuda")
    s.sgqa_paged_attn(pp, Q, Kp, Vp, table, q_start, dev(after).int(), O, lse,
                      s.alloc_paged_workspace(pp), status=st)
    assert status_of(s, st) == s.OK
    big = max(after)
    K, V = np.zeros((N, hk, big, d)), np.zeros((N, hk, big, d))
    for i, n in enumerate(after):
        for X, k in ((K, "K"), (V, "V")):
            X[i, :, :n] = synth.widen(inp[i][k]).transpose(1, 0, 2)[:, :n]
    R, z, tO, tl, _ = ref.attention(Q[:N].double().cpu().numpy(), K, V, big, np.arange(N)[:, None],
                                    np.arange(N + 1), after, ref.default_scale(d), True, 0, True)
    assert (np.abs(O[:N].double().cpu().numpy() - R) <= tO).all()
    assert (np.abs(lse[:, :N].double().cpu().numpy() - z) <= tl).all()


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
