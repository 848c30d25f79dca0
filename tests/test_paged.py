"""Paged serving operators: page tables and slot maps, page release, K/V append
and ragged attention over the pool, against plain 64-bit forms (paged_ref)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import paged_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def s():
    from block_sparse_long_sgqa_gb300 import sgqa

    return sgqa


def params(s, **kw):
    base = dict(n_seqs=3, max_tokens=10, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16,
                n_pages=20, max_pages=4)
    base.update(kw)
    return s.paged_params(**base)


# ------------------------------------------------------------- host, no GPU
def test_struct_matches_header(s):
    text = open(os.path.join(ROOT, "include", "sgqa.h")).read()
    body = re.search(r"typedef struct sgqa_paged_params \{(.*?)\} sgqa_paged_params;", text,
                     re.S).group(1)
    fields = re.findall(r"^\s*(?:int32_t|float)\s+(\w+);", body, re.M)
    assert fields == [n for n, _ in s.PagedParams._fields_]
    assert ctypes.sizeof(s.PagedParams) == 4 * len(fields)


P = 0x1000  # an aligned address that nothing reads: every call below is refused first


def call_attn(s, p, Q=P, K=P, V=P, pt=P, qs=P, kv=P, O=P, lse=P, ws=P, ws_bytes=1 << 50):
    return s._lib.sgqa_paged_attn(ctypes.byref(p), Q, K, V, pt, qs, kv, O, lse, ws, ws_bytes,
                                  None, None)


BAD_PARAMS = [
    (dict(n_seqs=-1), "INVALID_ARG"), (dict(max_tokens=-1), "INVALID_ARG"),
    (dict(n_pages=0), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
    (dict(page_size=0), "INVALID_ARG"), (dict(page_size=-8), "INVALID_ARG"),
    (dict(n_q_heads=7), "INVALID_ARG"), (dict(n_kv_heads=0), "INVALID_ARG"),
    (dict(n_q_heads=0), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"),
    (dict(causal=2), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(window=5, causal=0), "INVALID_ARG"),
    (dict(softmax_scale=-1.0), "INVALID_ARG"), (dict(softmax_scale=float("nan")), "INVALID_ARG"),
    (dict(softmax_scale=float("inf")), "INVALID_ARG"),
    (dict(q_stride=8), "INVALID_ARG"), (dict(kv_stride=-128), "INVALID_ARG"),
    (dict(head_dim=96), "UNSUPPORTED"), (dict(page_size=12), "UNSUPPORTED"),
    (dict(n_q_heads=258), "UNSUPPORTED"), (dict(max_tokens=(1 << 24) + 1), "UNSUPPORTED"),
    (dict(softmax_scale=3e38), "INVALID_ARG"),
    (dict(max_pages=(1 << 21) + 1), "UNSUPPORTED"),
    (dict(max_tokens=1 << 20, n_q_heads=2048, n_kv_heads=16), "UNSUPPORTED"), (dict(n_pages=1 << 27), "UNSUPPORTED"),
    (dict(q_stride=513), "ALIGNMENT"), (dict(kv_stride=130), "ALIGNMENT"),
]


@pytest.mark.parametrize("kw,code", BAD_PARAMS, ids=[str(k) for k, _ in BAD_PARAMS])
def test_bad_params_refused_by_every_entry(s, kw, code):
    causal = kw.get("causal", 1)
    p = params(s, **{k: v for k, v in kw.items() if k != "causal"})
    p.causal = causal
    want = getattr(s, "ERR_" + code)
    b = ctypes.byref(p)
    assert call_attn(s, p) == want
    assert s._lib.sgqa_page_plan(b, *[P + 16 * i for i in range(9)], None, None) == want
    assert s._lib.sgqa_page_release(b, *[P + 16 * i for i in range(6)], None, None) == want
    assert s._lib.sgqa_paged_append(b, P, P, P, P, P, None, None) == want
    assert s.paged_workspace_bytes(p) == 0


def test_bad_pointers_refused(s):
    p = params(s)
    for name in ("Q", "K", "V", "pt", "qs", "kv", "O", "lse"):
        assert call_attn(s, p, **{name: None}) == s.ERR_INVALID_ARG, name
    for name in ("Q", "K", "V", "O"):
        assert call_attn(s, p, **{name: P + 8}) == s.ERR_ALIGNMENT, name
    assert call_attn(s, p, ws=None) == s.ERR_WORKSPACE
    assert call_attn(s, p, ws_bytes=s.paged_workspace_bytes(p) - 1) == s.ERR_WORKSPACE
    b = ctypes.byref(p)
    plan, rel, app = s._lib.sgqa_page_plan, s._lib.sgqa_page_release, s._lib.sgqa_paged_append
    for i in range(9):
        args = [P + 16 * k for k in range(9)]
        args[i] = None
        assert plan(b, *args, None, None) == s.ERR_INVALID_ARG, i
    args = [P + 16 * k for k in range(9)]
    args[8] = args[3]  # n_free_out is n_free
    assert plan(b, *args, None, None) == s.ERR_INVALID_ARG
    for i in range(6):
        args = [P + 16 * k for k in range(6)]
        args[i] = None
        assert rel(b, *args, None, None) == s.ERR_INVALID_ARG, i
    args = [P + 16 * k for k in range(6)]
    args[5] = args[4]
    assert rel(b, *args, None, None) == s.ERR_INVALID_ARG
    for i in range(5):
        args = [P] * 5
        args[i] = None
        assert app(b, *args, None, None) == s.ERR_INVALID_ARG, i
        if i != 2:
            args[i] = P + 8
            assert app(b, *args, None, None) == s.ERR_ALIGNMENT, i


def test_empty_calls_enqueue_nothing(s):
    for kw in (dict(n_seqs=0), dict(max_tokens=0)):
        assert call_attn(s, params(s, **kw), Q=None, ws=None) == s.OK
    p = params(s, max_tokens=0)
    assert s._lib.sgqa_paged_append(ctypes.byref(p), None, None, None, P, P, None, None) == s.OK


def test_binding_refuses_wrong_tensors(s):
    """Shapes, types, strides and CPU tensors are turned away before the call."""
    p = params(s)
    i32 = dict(dtype=torch.int32)
    ok = dict(Q=torch.zeros(10, 8, 64, dtype=torch.bfloat16),
              K_pages=torch.zeros(20, 2, 16, 64, dtype=torch.bfloat16),
              V_pages=torch.zeros(20, 2, 16, 64, dtype=torch.bfloat16),
              page_table=torch.zeros(3, 4, **i32), q_start=torch.zeros(4, **i32),
              kv_len=torch.zeros(3, **i32), O=torch.zeros(10, 8, 64, dtype=torch.bfloat16),
              lse=torch.zeros(8, 10), ws=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        s.sgqa_paged_attn(p, **ok)
    bad = dict(Q=torch.zeros(10, 8, 64), K_pages=torch.zeros(19, 2, 16, 64, dtype=torch.bfloat16),
               page_table=torch.zeros(3, 4, dtype=torch.int64), q_start=torch.zeros(3, **i32),
               kv_len=torch.zeros(2, **i32), O=torch.zeros(10, 64, 8, dtype=torch.bfloat16).mT,
               lse=torch.zeros(8, 9))
    for k, v in bad.items():
        with pytest.raises(ValueError, match=k):
            s.sgqa_paged_attn(p, **{**ok, k: v})
    wide = torch.zeros(10, 12, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="strides"):
        s.sgqa_paged_attn(p, **{**ok, "Q": wide[:, :8]})
    with pytest.raises(ValueError, match="CUDA"):  # the same rows with the stride in the params
        s.sgqa_paged_attn(params(s, q_stride=12 * 64), **{**ok, "Q": wide[:, :8]})


# --------------------------------------------------------------------- pages
def dev(x, dtype=None):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def status_of(s, st):
    return s.read_status(st)[0]


class Batch:
    """A batch's tables on the host: pages dealt from a permutation."""

    def __init__(self, seed, q_len, kv_len, ps, spare=5, extra_cols=2, held_at="before"):
        rng = np.random.default_rng(seed)
        self.q, self.kv = np.array(q_len, np.int32), np.array(kv_len, np.int32)
        self.N, self.ps = len(q_len), ps
        self.max_pages = max([1] + [ref.pages_of(int(x), ps) for x in kv_len]) + extra_cols
        self.n_pages = sum(ref.pages_of(int(x), ps) for x in kv_len) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        before = self.kv - (self.q if held_at == "before" else 0)
        self.table = rng.integers(-(1 << 30), 1 << 30, (max(self.N, 1), self.max_pages),
                                  dtype=np.int32)  # garbage behind the pages held
        at = 0
        for i in range(self.N):
            n = ref.pages_of(int(before[i]), ps)
            self.table[i, :n] = order[at:at + n]
            at += n
        self.free = np.full(self.n_pages, -7, np.int32)
        self.n_free = self.n_pages - at
        self.free[:self.n_free] = order[at:]


PLANS = {
    "decode": ([1] * 9, [1, 16, 17, 32, 33, 5, 48, 49, 64], 16, 0),
    "one": ([1], [1], 8, 0),
    "chunk": ([100, 0, 1, 37, 0, 64], [100, 50, 51, 101, 0, 128], 16, 30),
    "idle_ends": ([0, 0, 3, 0, 0], [0, 9, 8, 7, 0], 8, 1),
    "page_24": ([50, 7, 24], [70, 7, 48], 24, 0),
    "none": ([0, 0], [0, 40], 16, 4),
    "long": ([1500, 1], [1500, 3000], 64, 100),
    # more requests than are summed at a time (2048), most of them idle or single tokens
    "many": ([i % 3 for i in range(5000)], [i % 3 + i % 40 for i in range(5000)], 8, 11),
}


def run_plan(s, b, pad, **over):
    T = int(b.q.sum()) + pad
    a = dict(q_len=dev(b.q), kv_len=dev(b.kv), free_pages=dev(b.free), n_free=dev([b.n_free]),
             page_table=dev(b.table))
    a = {k: v.to(torch.int32) for k, v in a.items()}
    for k, v in over.items():
        a[k] = dev(v).to(torch.int32)
    p = params(s, n_seqs=b.N, max_tokens=over.pop("T", T) if "T" in over else T, page_size=b.ps,
               n_pages=b.n_pages, max_pages=b.max_pages)
    out = dict(q_start=torch.full((b.N + 3,), 77, dtype=torch.int32).cuda(),
               slot_map=torch.full((T + 2,), 77, dtype=torch.int64).cuda(),
               positions=torch.full((T + 2,), 77, dtype=torch.int32).cuda(),
               n_free_out=torch.full((1,), 77, dtype=torch.int32).cuda())
    st = s.new_status()
    s.sgqa_page_plan(p, **a, **out, status=st)
    code = status_of(s, st)
    return p, a, {k: v.cpu().numpy() for k, v in out.items()}, code


@gpu
@pytest.mark.parametrize("name", PLANS)
def test_plan(s, name):
    q, kv, ps, pad = PLANS[name]
    b = Batch(1, q, kv, ps)
    p, a, out, code = run_plan(s, b, pad)
    assert code == s.OK
    T = p.max_tokens
    table, q_start, slots, pos, n_free = ref.plan(q, kv, b.free, b.n_free, b.table, ps, T)
    assert np.array_equal(a["page_table"].cpu().numpy(), table)
    assert np.array_equal(out["q_start"][:b.N + 1], q_start) and (out["q_start"][b.N + 1:] == 77).all()
    assert np.array_equal(out["slot_map"][:T], slots) and (out["slot_map"][T:] == 77).all()
    assert np.array_equal(out["positions"][:T], pos) and (out["positions"][T:] == 77).all()
    assert out["n_free_out"][0] == n_free
    assert np.array_equal(a["free_pages"].cpu().numpy(), b.free)


@gpu
@pytest.mark.parametrize("what", ["pages", "tokens", "negative", "short", "long", "n_free"])
@pytest.mark.parametrize("many", [False, True])
def test_plan_that_does_not_fit_takes_nothing(s, what, many):
    q, kv, ps, pad = PLANS["many" if many else "chunk"]
    b = Batch(2, q, kv, ps, spare=0)
    over, want = {}, s.ERR_BOUNDS
    k = b.N - 2
    if what == "pages":
        over["n_free"], want = [b.n_free - 1], s.ERR_CAPACITY
    elif what == "tokens":
        q2, kv2 = b.q.copy(), b.kv.copy()
        q2[k] += pad + 1
        kv2[k] += pad + 1
        b.max_pages += 8
        b.table = np.concatenate([b.table, np.zeros((b.N, 8), np.int32)], 1)
        over.update(q_len=q2, kv_len=kv2)
        want = s.ERR_CAPACITY
    elif what == "negative":
        q2 = b.q.copy()
        q2[k] = -1
        over["q_len"] = q2
    elif what == "short":
        kv2 = b.kv.copy()
        kv2[k] = b.q[k] - 1
        over["kv_len"] = kv2
    elif what == "long":
        kv2 = b.kv.copy()
        kv2[k] = b.max_pages * ps + 1
        over["kv_len"] = kv2
    else:
        over["n_free"] = [b.n_pages + 1]
    p, a, out, code = run_plan(s, b, pad, **over)
    assert code == want
    assert np.array_equal(a["page_table"].cpu().numpy(), b.table)
    assert (out["q_start"][:b.N + 1] == 0).all()
    assert (out["slot_map"][:p.max_tokens] == -1).all() and (out["positions"][:p.max_tokens] == -1).all()
    assert out["n_free_out"][0] == a["n_free"].item()


@gpu
def test_plan_page_outside_the_pool(s):
    """A held page number outside the pool gives its tokens no slot."""
    b = Batch(3, [1, 1], [5, 6], 16)
    b.table[1, 0] = b.n_pages
    _, _, out, code = run_plan(s, b, 0)
    assert code == s.ERR_BOUNDS
    assert out["slot_map"][1] == -1 and out["slot_map"][0] == b.table[0, 0] * 16 + 4


@gpu
@pytest.mark.parametrize("n,ps", [(1, 8), (5, 16), (300, 24), (4500, 8)])
def test_release(s, n, ps):
    rng = np.random.default_rng(n)
    kv = rng.integers(0, 200, n)
    keep = np.where(rng.random(n) < 0.5, 0, rng.integers(0, kv + 1))
    b = Batch(4, [0] * n, kv, ps, held_at="after")
    p = params(s, n_seqs=n, max_tokens=0, page_size=ps, n_pages=b.n_pages, max_pages=b.max_pages)
    free, nf = dev(b.free), dev([b.n_free]).to(torch.int32)
    out, st = torch.zeros_like(nf), s.new_status()
    s.sgqa_page_release(p, dev(kv).to(torch.int32), dev(keep).to(torch.int32), dev(b.table), free,
                        nf, out, status=st)
    want, n_free = ref.release(kv, keep, b.table, b.free, b.n_free, ps)
    assert status_of(s, st) == s.OK
    assert np.array_equal(free.cpu().numpy(), want) and out.item() == n_free


@gpu
@pytest.mark.parametrize("what", ["keep", "negative", "full"])
def test_release_refused_changes_nothing(s, what):
    kv, keep = np.array([40, 33]), np.array([0, 20])
    b = Batch(5, [0, 0], kv, 16, held_at="after")
    n_free = b.n_free
    if what == "keep":
        keep[1] = 34
    elif what == "negative":
        keep[0] = -1
    else:
        n_free = b.n_pages - 1
    p = params(s, n_seqs=2, max_tokens=0, page_size=16, n_pages=b.n_pages, max_pages=b.max_pages)
    free, nf = dev(b.free), dev([n_free]).to(torch.int32)
    out, st = torch.zeros_like(nf), s.new_status()
    s.sgqa_page_release(p, dev(kv).to(torch.int32), dev(keep).to(torch.int32), dev(b.table), free,
                        nf, out, status=st)
    assert status_of(s, st) == (s.ERR_CAPACITY if what == "full" else s.ERR_BOUNDS)
    assert np.array_equal(free.cpu().numpy(), b.free) and out.item() == n_free


# -------------------------------------------------------------------- append
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,hk,d,ps,fused", [(1, 1, 64, 8, False), (77, 8, 128, 64, True),
                                             (130, 3, 64, 24, True), (1000, 5, 128, 16, False)])
def test_append(s, dtype, T, hk, d, ps, fused):
    """Rows land bit for bit where their slots say, the rest of the pool stays,
    rows without a slot and slots outside the pool are skipped."""
    rng = np.random.default_rng(T)
    n_pages = ref.pages_of(T, ps) + 3
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    it = torch.int16 if dtype == "bf16" else torch.int32
    info = torch.iinfo(it)
    # any bit patterns, NaN and infinities among them
    def bits(*shape):
        return torch.from_numpy(rng.integers(info.min, info.max, shape)).to(it).cuda()

    width = (2 * hk + 3) * d if fused else hk * d
    x = bits(T, width)
    K, V = (x[:, d:(hk + 1) * d], x[:, (hk + 1) * d:(2 * hk + 1) * d]) if fused else (x, bits(T, width))
    K, V = (y.view(dt).unflatten(1, (hk, d)) for y in (K, V))
    Kp, Vp = bits(n_pages, hk, ps, d), bits(n_pages, hk, ps, d)
    slots = rng.permutation(n_pages * ps)[:T].astype(np.int64)
    if T > 10:
        slots[[3, 5]] = -1, -(1 << 40)
    p = params(s, max_tokens=T, n_q_heads=hk, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=n_pages, dtype=s.BF16 if dtype == "bf16" else s.FP32,
               kv_stride=width if fused else 0)
    want = [Kp.cpu().numpy().copy(), Vp.cpu().numpy().copy()]
    for t, at in enumerate(slots):
        if at >= 0:
            for w, y in zip(want, (K, V)):
                w[at // ps, :, at % ps] = y[t].contiguous().view(it).cpu().numpy()
    st = s.new_status()
    s.sgqa_paged_append(p, K, V, dev(slots), Kp.view(dt), Vp.view(dt), status=st)
    assert status_of(s, st) == s.OK
    assert np.array_equal(Kp.cpu().numpy(), want[0]) and np.array_equal(Vp.cpu().numpy(), want[1])
    if T > 10:
        slots[7] = n_pages * ps
        s.sgqa_paged_append(p, K, V, dev(slots), Kp.view(dt), Vp.view(dt), status=st)
        assert status_of(s, st) == s.ERR_BOUNDS
        assert np.array_equal(Kp.cpu().numpy(), want[0]) and np.array_equal(Vp.cpu().numpy(), want[1])


# ----------------------------------------------------------------- attention
# name: (q_len, kv_len, H, Hkv, d, page, kwargs)
ATTN = {
    "one_token": ([1], [1], 8, 2, 64, 16, {}),
    "decode": ([1] * 7, [1, 127, 128, 129, 300, 0, 511], 32, 4, 128, 64, {}),
    "decode_long": ([1], [9000], 16, 2, 128, 64, {}),
    "decode_d64": ([1, 1, 1], [700, 64, 3], 8, 8, 64, 8, {}),
    "decode_g128": ([1, 1], [200, 77], 128, 1, 64, 16, {}),
    "drafts": ([5, 2, 9], [405, 130, 9], 16, 2, 128, 16, {}),
    "drafts_g7": ([3, 4, 18], [500, 129, 150], 28, 4, 128, 32, {}),
    "prompt": ([200], [200], 8, 1, 128, 64, {}),
    "prompt_g1": ([300, 131], [300, 131], 3, 3, 64, 128, {}),
    "chunk": ([130, 64], [1000, 321], 16, 2, 128, 16, {}),
    "chunk_g3": ([90, 1, 45], [190, 700, 45], 6, 2, 64, 24, {}),
    "mixed_idle": ([0, 100, 1, 0, 33, 1], [50, 100, 1025, 0, 290, 1], 16, 4, 128, 16, {}),
    "big_pages": ([40, 1], [600, 513], 8, 2, 128, 256, {}),
    "page_40": ([33, 1], [260, 1000], 8, 2, 64, 40, {}),
    "window": ([150, 1, 20], [400, 900, 20], 8, 2, 128, 16, dict(window=100)),
    "window_1": ([40, 1], [140, 500], 8, 1, 64, 16, dict(window=1)),
    "window_decode": ([1, 1, 1], [5000, 128, 300], 16, 2, 128, 64, dict(window=128)),
    "window_wide": ([70], [300], 8, 2, 128, 64, dict(window=100000)),
    "full": ([50, 1, 7, 3], [260, 33, 0, 128], 8, 2, 128, 16, dict(causal=False)),
    "below_zero": ([6, 200], [2, 100], 8, 2, 64, 16, {}),
    "scale": ([9, 1], [100, 222], 8, 2, 64, 16, dict(softmax_scale=0.5)),
    "padding": ([3, 1], [40, 200], 8, 2, 128, 16, dict(pad=70)),
    "fused_rows": ([20, 1], [150, 33], 8, 2, 64, 16, dict(fused=True)),
    # one request over every CTA, and more requests than threads look at first
    "decode_split": ([1], [30000], 1, 1, 128, 64, {}),
    "decode_split_16": ([1], [20011], 16, 1, 64, 32, {}),
    "many_requests": ([1, 0, 1] * 150, [(7 * i) % 131 + 1 for i in range(450)], 4, 2, 64, 16, {}),
    "many_chunks": ([1, 40, 0, 17] * 20, [60 + 31 * (i % 9) for i in range(80)], 8, 2, 64, 16, {}),
    "one_head_many_tiles": ([1000], [1300], 4, 1, 64, 32, {}),
    # few rows a request, one of them with all the tokens, two tokens an item
    "few_g5": ([1, 1, 1], [3000, 95, 97], 20, 4, 128, 16, {}),
    "few_g8_d64": ([1] * 5, [1, 63, 64, 65, 2000], 16, 2, 64, 8, {}),
    "few_g16": ([1] * 4, [96, 191, 193, 2500], 32, 2, 128, 64, {}),
    "few_g11_window": ([1, 1], [1500, 30], 22, 2, 64, 24, dict(window=70)),
    "few_in_one_request": ([6, 0, 0, 0, 0, 0], [500, 9, 0, 3, 0, 1], 16, 2, 128, 16, {}),
    "few_two_tokens": ([2, 2, 2], [300, 100, 2], 8, 2, 128, 40, {}),
    "few_full": ([1, 1], [700, 0], 16, 2, 128, 16, dict(causal=False)),
}


def attn_case(s, name, dtype, spread=1.0, garbage=True):
    q_len, kv_len, H, hk, d, ps, kw = ATTN[name]
    kw = dict(kw)
    pad, fused = kw.pop("pad", 0), kw.pop("fused", False)
    b = Batch(6, q_len, kv_len, ps, held_at="after")
    T = int(b.q.sum()) + pad
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(len(name) * 100 + d)
    wide = torch.randn(T, H + 2 * hk if fused else H, d, generator=g).mul_(spread).to(dt)
    K = torch.randn(b.n_pages, hk, ps, d, generator=g).to(dt)
    V = torch.randn(b.n_pages, hk, ps, d, generator=g).to(dt)
    if garbage:  # what no position of the batch holds
        used = np.zeros((b.n_pages, ps), bool)
        for i in range(b.N):
            for j in range(int(b.kv[i])):
                used[b.table[i, j // ps], j % ps] = True
        free = torch.from_numpy(~used)[:, None, :, None].expand_as(K)
        K[free] = float("nan")
        V[free] = float("nan")
        V.view(-1)[::7][free.reshape(-1)[::7]] = float("inf")
    p = params(s, n_seqs=b.N, max_tokens=T, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=b.n_pages, max_pages=b.max_pages,
               dtype=s.BF16 if dtype == "bf16" else s.FP32,
               q_stride=(H + 2 * hk) * d if fused else 0, **kw)
    q_start = np.concatenate([[0], np.cumsum(b.q)]).astype(np.int32)
    return b, p, wide, K, V, q_start, kw


def run_attn(s, p, wide, K, V, table, q_start, kv, ws=None):
    O = torch.full((p.max_tokens, p.n_q_heads, p.head_dim), 3.0, dtype=wide.dtype).cuda()
    lse = torch.full((p.n_q_heads, p.max_tokens), 7.0).cuda()
    ws = s.alloc_paged_workspace(p) if ws is None else ws
    ws.fill_(0xFF)  # NaN wherever the workspace is read unwritten
    st = s.new_status()
    s.sgqa_paged_attn(p, wide.cuda()[:, :p.n_q_heads], K.cuda(), V.cuda(), dev(table),
                      dev(q_start), dev(kv), O, lse, ws, status=st)
    return O, lse, status_of(s, st)


def f64(x):
    return np.nan_to_num(x.double().numpy(), nan=1e30, posinf=1e30)


def check_attn(s, b, p, wide, K, V, q_start, kw, O, lse):
    H, d = p.n_q_heads, p.head_dim
    bf16 = p.dtype == s.BF16
    R, z, tO, tl, mine = ref.attention(
        wide[:, :H].double().numpy(), f64(K), f64(V), b.ps, b.table, q_start, b.kv,
        kw.get("softmax_scale") or ref.default_scale(d), kw.get("causal", True),
        kw.get("window", 0), bf16)
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (O[~mine] == 3.0).all() and (lse[:, ~mine] == 7.0).all()  # padding rows left alone
    assert np.isfinite(O).all()
    over = np.abs(O - R)[mine] - tO[mine]
    assert over.size == 0 or over.max() <= 0, (over.max(), np.abs(O - R)[mine].max())
    seen = np.isfinite(z)
    assert np.array_equal(np.isneginf(lse)[:, mine], ~seen[:, mine])
    with np.errstate(invalid="ignore"):
        dl = np.abs(lse - z) - tl
    assert not mine.any() or not (seen & mine).any() or dl[seen & mine].max() <= 0, dl[seen & mine].max()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", ATTN)
def test_attention(s, name, dtype):
    """Against the 64-bit form; the pool holds NaN and infinities wherever no
    position of the batch lies, the page table garbage behind the pages."""
    b, p, wide, K, V, q_start, kw = attn_case(s, name, dtype)
    O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    assert code == s.OK
    check_attn(s, b, p, wide, K, V, q_start, kw, O, lse)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", ["decode", "chunk", "window"])
def test_attention_peaked(s, name, dtype):
    """Logits of standard deviation 12: the running maximum climbs by far more
    than a tile's weights can hold, in both halves of tiles."""
    b, p, wide, K, V, q_start, kw = attn_case(s, name, dtype, spread=12.0)
    O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    assert code == s.OK
    check_attn(s, b, p, wide, K, V, q_start, kw, O, lse)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", ["decode", "decode_split_16", "few_g16", "chunk", "mixed_idle"])
def test_attention_nan_stays_with_its_rows(s, name, dtype):
    """A NaN key makes the rows that see it NaN, in O and lse, whole or cut items
    alike; other requests and other heads keep their bits."""
    b, p, wide, K, V, q_start, kw = attn_case(s, name, dtype)
    O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    assert code == s.OK
    i = int(np.argmax(b.kv * (b.q > 0)))
    pos, g, G = int(b.kv[i] - b.q[i]) // 2, p.n_kv_heads - 1, p.n_q_heads // p.n_kv_heads
    K[b.table[i, pos // b.ps], g, pos % b.ps, 5] = float("nan")
    On, ln, code = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    assert code == s.OK
    rows = torch.zeros(p.max_tokens, dtype=torch.bool)
    rows[q_start[i]:q_start[i + 1]] = True
    heads = torch.zeros(p.n_q_heads, dtype=torch.bool)
    heads[g * G:(g + 1) * G] = True
    hit = (rows[:, None] & heads[None, :]).cuda()
    assert torch.isnan(On[hit]).all() and torch.isnan(ln.T[hit]).all()
    assert torch.equal(On[~hit], O[~hit]) and torch.equal(ln.T[~hit], lse.T[~hit])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_repeats_bit_for_bit(s, dtype):
    for name in ("decode_long", "mixed_idle", "chunk"):
        b, p, wide, K, V, q_start, kw = attn_case(s, name, dtype)
        a = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
        c = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_bad_tables(s, dtype):
    """Page numbers outside the pool read as zeros and are reported; bad
    lengths and row ranges drop their request and leave the others right."""
    b, p, wide, K, V, q_start, kw = attn_case(s, "chunk", dtype)
    for bad in (-1, b.n_pages, -(1 << 31), (1 << 31) - 1):
        table = b.table.copy()
        table[0, 3] = bad
        _, _, code = run_attn(s, p, wide, K, V, table, q_start, b.kv)
        assert code == s.ERR_BOUNDS
    for kv0 in (-1, p.max_pages * b.ps + 1, (1 << 31) - 1, -(1 << 31)):
        kv = b.kv.copy()
        kv[0] = kv0
        O, lse, code = run_attn(s, p, wide, K, V, b.table, q_start, kv)
        assert code == s.ERR_BOUNDS
        n = int(b.q[0])
        assert (O[:n] == 3.0).all() and (lse[:, :n] == 7.0).all()
        ok, ok_lse, _ = run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
        assert torch.isfinite(O[n:].float()).all()
        assert (O[n:] - ok[n:]).abs().max() < 0.05  # the split of the keys may differ
    for row in ([0, 130, 129], [5, 2, 194], [-3, 130, 194], [0, 130, 195], [0, 1 << 30, 194]):
        _, _, code = run_attn(s, p, wide, K, V, b.table, np.array(row, np.int32), b.kv)
        assert code == s.ERR_BOUNDS


@gpu
def test_attention_other_stream(s):
    """The call runs on the stream it is given, behind that stream's work."""
    b, p, wide, K, V, q_start, kw = attn_case(s, "drafts", "bf16")
    st = torch.cuda.Stream()
    Q = wide.cuda()
    Kd, Vd = torch.zeros_like(K, device="cuda"), torch.zeros_like(V, device="cuda")
    Ks, Vs = K.cuda(), V.cuda()
    O = torch.full(Q.shape, 3.0, dtype=Q.dtype, device="cuda")
    lse = torch.full((p.n_q_heads, p.max_tokens), 7.0, device="cuda")
    ws = s.alloc_paged_workspace(p)
    pt, qs, kv = dev(b.table), dev(q_start), dev(b.kv)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        Kd.copy_(Ks)
        Vd.copy_(Vs)
    s.sgqa_paged_attn(p, Q, Kd, Vd, pt, qs, kv, O, lse, ws, stream=st)
    st.synchronize()
    check_attn(s, b, p, wide, K, V, q_start, kw, O, lse)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_waves(s, dtype):
    """Two requests whose shared keys exceed what L2 holds: whole items go out in
    waves first, the rest of each request evenly; checked on spread rows."""
    d, hk, ps = 128, 8, 64
    H = 64 if dtype == "bf16" else 16
    b = Batch(8, [700, 650], [20011, 15000], ps, held_at="after")
    T = 1350
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    p = params(s, n_seqs=2, max_tokens=T, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=b.n_pages, max_pages=b.max_pages,
               dtype=s.BF16 if dtype == "bf16" else s.FP32)
    torch.manual_seed(3)
    Q = torch.randn(T, H, d, device="cuda").to(dt)
    K, V = (torch.randn(b.n_pages, hk, ps, d, device="cuda").to(dt) for _ in "KV")
    q_start = np.array([0, 700, 1350], np.int32)
    O, lse, code = run_attn(s, p, Q.cpu(), K, V, b.table, q_start, b.kv)
    assert code == s.OK
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(O).all() and np.isfinite(lse).all()
    Kn, Vn, Qn = (x.double().cpu().numpy() for x in (K, V, Q))
    for r in range(2):
        for i in (0, 1, 31, 32, 333, int(b.q[r]) - 1):  # one row as a batch of its own
            t = int(q_start[r]) + i
            n = int(b.kv[r] - b.q[r]) + i + 1
            R, z, tO, tl, _ = ref.attention(Qn[t:t + 1], Kn, Vn, ps, b.table[r:r + 1],
                                            [0, 1], [n], ref.default_scale(d), True, 0,
                                            dtype == "bf16")
            assert (np.abs(O[t] - R[0]) <= tO[0]).all(), (r, i)
            assert (np.abs(lse[:, t] - z[:, 0]) <= tl[:, 0]).all(), (r, i)


@gpu
def test_offsets_past_4_gib(s):
    """Pages at the far end of a pool of more than 4 GiB: rows appended there are
    found by the attention, and nothing else of the pool is touched."""
    d, hk, H, ps, n_pages = 128, 8, 16, 64, 40000   # 5.2 GB for K, as much for V
    p = params(s, n_seqs=1, max_tokens=150, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=n_pages, max_pages=3)
    Kp, Vp = (torch.zeros(n_pages, hk, ps, d, dtype=torch.bfloat16, device="cuda") for _ in "KV")
    torch.manual_seed(4)
    Q = torch.randn(150, H, d, device="cuda").bfloat16()
    K, V = (torch.randn(150, hk, d, device="cuda").bfloat16() for _ in "KV")
    table = np.array([[n_pages - 1, 2, n_pages - 2]], np.int32)
    pos = np.arange(150)
    slots = table[0, pos // ps].astype(np.int64) * ps + pos % ps
    st = s.new_status()
    s.sgqa_paged_append(p, K, V, dev(slots), Kp, Vp, status=st)
    O, lse = torch.zeros_like(Q), torch.zeros(H, 150, device="cuda")
    s.sgqa_paged_attn(p, Q, Kp, Vp, dev(table), dev(np.array([0, 150], np.int32)),
                      dev(np.array([150], np.int32)), O, lse, s.alloc_paged_workspace(p), status=st)
    assert status_of(s, st) == s.OK
    assert torch.equal(Kp[n_pages - 1].transpose(0, 1), K[:64])
    used = Kp.view(torch.int16).ne(0).flatten(1).any(1).nonzero().flatten().tolist()
    assert used == [2, n_pages - 2, n_pages - 1]
    Kl, Vl = (x.double().cpu().numpy().transpose(1, 0, 2)[None] for x in (K, V))
    R, z, tO, tl, _ = ref.attention(Q.double().cpu().numpy(), Kl, Vl, 150, np.zeros((1, 1), int),
                                    [0, 150], [150], ref.default_scale(d), True, 0, True)
    assert (np.abs(O.double().cpu().numpy() - R) <= tO).all()
    assert (np.abs(lse.double().cpu().numpy() - z) <= tl).all()


@gpu
def test_attention_output_at_16_bytes(s):
    """O and Q that are 16-byte but not 32-byte aligned, rows before and behind kept."""
    b, p, wide, K, V, q_start, kw = attn_case(s, "chunk", "bf16")
    n = p.max_tokens * p.n_q_heads * p.head_dim
    raw = torch.full((n + 24,), 5.0, dtype=torch.bfloat16, device="cuda")
    O = raw[8:8 + n].view(p.max_tokens, p.n_q_heads, p.head_dim)
    q_raw = torch.zeros(n + 8, dtype=torch.bfloat16, device="cuda")
    q_raw[8:] = wide.cuda().flatten()
    Q = q_raw[8:].view_as(O)
    assert O.data_ptr() % 32 == 16 and Q.data_ptr() % 32 == 16
    lse = torch.full((p.n_q_heads, p.max_tokens), 7.0).cuda()
    s.sgqa_paged_attn(p, Q, K.cuda(), V.cuda(), dev(b.table), dev(q_start), dev(b.kv), O, lse,
                      s.alloc_paged_workspace(p))
    check_attn(s, b, p, wide, K, V, q_start, kw, O, lse)
    assert (raw[:8] == 5.0).all() and (raw[8 + n:] == 5.0).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_graphs_share_a_workspace(s, dtype):
    """Two captured calls of different shapes over one workspace, replayed in turn
    and with other lengths, give what the same calls give eagerly on their own."""
    cases, graphs = [], []
    parts = [attn_case(s, name, dtype) for name in ("decode_long", "mixed_idle")]
    ws = torch.empty(max(s.paged_workspace_bytes(c[1]) for c in parts), dtype=torch.uint8,
                     device="cuda")
    for b, p, wide, K, V, q_start, kw in parts:
        t = dict(Q=wide.cuda(), K_pages=K.cuda(), V_pages=V.cuda(), page_table=dev(b.table),
                 q_start=dev(q_start), kv_len=dev(b.kv))
        O = torch.full(wide.shape, 3.0, dtype=wide.dtype, device="cuda")
        lse = torch.full((p.n_q_heads, p.max_tokens), 7.0, device="cuda")
        s.sgqa_paged_attn(p, **t, O=O, lse=lse, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.sgqa_paged_attn(p, **t, O=O, lse=lse, ws=ws)
        cases.append((b, p, t, O, lse))
        graphs.append(g)
    for it in range(3):
        for g, (b, p, t, O, lse) in zip(graphs, cases):
            t["kv_len"].copy_(dev(np.maximum(b.kv - 3 * it, 0)))
            g.replay()
        for b, p, t, O, lse in cases:
            O2, l2 = torch.full_like(O, 3.0), torch.full_like(lse, 7.0)
            s.sgqa_paged_attn(p, **t, O=O2, lse=l2, ws=s.alloc_paged_workspace(p))
            assert torch.equal(O, O2) and torch.equal(lse, l2), it


@gpu
def test_attention_captured_behind_copies(s):
    """A captured step whose inputs come by copies and fills inside the graph."""
    b, p, wide, K, V, q_start, kw = attn_case(s, "chunk", "bf16")
    src = [wide.cuda(), dev(b.kv)]
    Q, kv = torch.zeros_like(src[0]), torch.zeros_like(src[1])
    Kd, Vd, pt, qs = K.cuda(), V.cuda(), dev(b.table), dev(q_start)
    O = torch.zeros_like(Q)
    lse = torch.zeros(p.n_q_heads, p.max_tokens, device="cuda")
    ws = s.alloc_paged_workspace(p)

    def step():
        Q.copy_(src[0])
        kv.copy_(src[1])
        O.zero_()
        s.sgqa_paged_attn(p, Q, Kd, Vd, pt, qs, kv, O, lse, ws)
        Q.zero_()
        kv.zero_()

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(5):
        O.fill_(9.0)
        lse.fill_(9.0)
        g.replay()
        check_attn(s, b, p, wide, K, V, q_start, kw, O, lse)


@gpu
def test_attention_calls_at_once(s):
    """Calls on two streams with a workspace each."""
    outs = []
    work = [attn_case(s, name, "bf16") for name in ("chunk", "decode_long")]
    args = []
    for b, p, wide, K, V, q_start, kw in work:
        args.append(dict(Q=wide.cuda(), K_pages=K.cuda(), V_pages=V.cuda(),
                         page_table=dev(b.table), q_start=dev(q_start), kv_len=dev(b.kv),
                         O=torch.full(wide.shape, 3.0, dtype=wide.dtype, device="cuda"),
                         lse=torch.full((p.n_q_heads, p.max_tokens), 7.0, device="cuda"),
                         ws=s.alloc_paged_workspace(p)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(20):
        for w, a, st in zip(work, args, streams):
            s.sgqa_paged_attn(w[1], **a, stream=st)
    torch.cuda.synchronize()
    for (b, p, wide, K, V, q_start, kw), a in zip(work, args):
        check_attn(s, b, p, wide, K, V, q_start, kw, a["O"], a["lse"])


@gpu
def test_stalled_wait_reports_timeout_and_recovers(s):
    """The debug request of the status word makes the first piece's pipeline give up
    after 1 ms: the status says so, and the next call on the same buffers is right."""
    b, p, wide, K, V, q_start, kw = attn_case(s, "chunk", "bf16")
    a = dict(Q=wide.cuda(), K_pages=K.cuda(), V_pages=V.cuda(), page_table=dev(b.table),
             q_start=dev(q_start), kv_len=dev(b.kv),
             O=torch.full(wide.shape, 3.0, dtype=wide.dtype, device="cuda"),
             lse=torch.full((p.n_q_heads, p.max_tokens), 7.0, device="cuda"),
             ws=s.alloc_paged_workspace(p))
    st = s.new_status()
    st[3] = s.DEBUG_STALL
    s.sgqa_paged_attn(p, **a, status=st)
    code, detail = s.read_status(st)
    assert code == s.ERR_TIMEOUT and detail == 220, (s.status_string(code), detail)
    s.reset_status(st)
    s.sgqa_paged_attn(p, **a, status=st)
    assert status_of(s, st) == s.OK
    check_attn(s, b, p, wide, K, V, q_start, kw, a["O"], a["lse"])


@gpu
def test_launch_log_names_the_kernels(s):
    b, p, wide, K, V, q_start, kw = attn_case(s, "chunk", "bf16")
    with s.launch_log(8) as log:
        run_attn(s, p, wide, K, V, b.table, q_start, b.kv)
    torch.cuda.synchronize()
    assert [k for k, _ in log.entries()] == [s.K_PAGED_ATTN] * 2  # the attention and its merge


# ------------------------------------------------------- the operators together
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(s, dtype, graph):
    """Requests come, grow by chunks and single tokens, drop drafted tokens and
    end, over one pool: each step plans its pages, appends its rows and attends;
    checked against the keys and values kept per request on the host.  With
    `graph` the three calls are captured once and replayed with new lengths."""
    rng = np.random.default_rng(11)
    g = torch.Generator().manual_seed(5)
    N, H, hk, d, ps, n_pages, T = 5, 8, 2, 64, 16, 90, 160
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    p = params(s, n_seqs=N, max_tokens=T, n_q_heads=H, n_kv_heads=hk, head_dim=d, page_size=ps,
               n_pages=n_pages, max_pages=30, dtype=s.BF16 if dtype == "bf16" else s.FP32,
               q_stride=(H + 2 * hk) * d, kv_stride=(H + 2 * hk) * d)
    i32 = dict(dtype=torch.int32, device="cuda")
    q_len, kv_len, keep = torch.zeros(N, **i32), torch.zeros(N, **i32), torch.zeros(N, **i32)
    free, nf, nf2 = dev(rng.permutation(n_pages)).to(torch.int32), torch.full((1,), n_pages, **i32), torch.zeros(1, **i32)
    table, q_start = torch.full((N, 30), -1, **i32), torch.zeros(N + 1, **i32)
    slots, pos = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(T, **i32)
    Kp, Vp = (torch.full((n_pages, hk, ps, d), float("nan"), dtype=dt, device="cuda") for _ in "kv")
    qkv = torch.zeros(T, H + 2 * hk, d, dtype=dt, device="cuda")
    O = torch.zeros(T, H, d, dtype=dt, device="cuda")
    lse = torch.zeros(H, T, device="cuda")
    ws, st = s.alloc_paged_workspace(p), s.new_status()

    def step():
        s.sgqa_page_plan(p, q_len, kv_len, free, nf, table, q_start, slots, pos, nf2, status=st)
        s.sgqa_paged_append(p, qkv[:, H:H + hk], qkv[:, H + hk:], slots, Kp, Vp, status=st)
        s.sgqa_paged_attn(p, qkv[:, :H], Kp, Vp, table, q_start, kv_len, O, lse, ws, status=st)

    run = step
    if graph:
        step()  # one eager run of empty requests
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
        run = cg.replay
    hist = [np.zeros((0, 2 * hk, d)) for _ in range(N)]
    for it in range(8):
        q = np.array([[100, 0, 1, 20, 7], [1, 30, 1, 1, 0], [1, 1, 60, 0, 3]][it % 3], np.int32)
        new = torch.randn(T, H + 2 * hk, d, generator=g).to(dt)
        kv = np.array([len(h) for h in hist], np.int32) + q
        qkv.copy_(new)
        q_len.copy_(torch.from_numpy(q))
        kv_len.copy_(torch.from_numpy(kv))
        O.fill_(3.0)
        lse.fill_(7.0)
        run()
        assert status_of(s, st) == s.OK
        nf.copy_(nf2)
        rows = new.double().numpy()
        t = 0
        for i in range(N):
            hist[i] = np.concatenate([hist[i], rows[t:t + q[i], H:]])
            t += q[i]
        # the same batch with one page per request, in order
        big = max(1, max(len(h) for h in hist))
        K, V = np.zeros((N, hk, big, d)), np.zeros((N, hk, big, d))
        for i, h in enumerate(hist):
            K[i, :, :len(h)], V[i, :, :len(h)] = h[:, :hk].transpose(1, 0, 2), h[:, hk:].transpose(1, 0, 2)
        qs = np.concatenate([[0], np.cumsum(q)])
        R, z, tO, tl, mine = ref.attention(rows[:, :H], K, V, big, np.arange(N)[:, None], qs, kv,
                                           ref.default_scale(d), True, 0, dtype == "bf16")
        Og, lg = O.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (np.abs(Og - R)[mine] <= tO[mine]).all()
        assert (np.abs(lg - z)[:, mine] <= tl[:, mine]).all()
        assert (Og[~mine] == 3.0).all() and (lg[:, ~mine] == 7.0).all()
        # one request ends, another takes its last tokens back
        left = kv.copy()
        left[it % N] = 0
        left[(it + 1) % N] = max(0, left[(it + 1) % N] - 5)
        keep.copy_(torch.from_numpy(left))
        s.sgqa_page_release(p, kv_len, keep, table, free, nf, nf2, status=st)
        assert status_of(s, st) == s.OK
        nf.copy_(nf2)
        hist = [h[:n] for h, n in zip(hist, left)]
        held = sum(ref.pages_of(int(n), ps) for n in left)
        assert nf.item() == n_pages - held
        # every page is free or held, once
        owned = table.cpu().numpy()
        owned = np.concatenate([owned[i, :ref.pages_of(int(n), ps)] for i, n in enumerate(left)])
        assert sorted(np.concatenate([owned, free.cpu().numpy()[:nf.item()]]).tolist()) == list(range(n_pages))
