"""The paged-cache operators of a round against the float64 oracle, through the C-ABI.

Whole numbers and copies must be equal.  The attention's tolerances, per element,
with A = sum_p w_p |v_p| / sum_p w_p from the oracle and u = 2^-9 (bf16's half step):
  out: u |out| for its own rounding + u A for the weights rounded to bf16, and
       2e-4 A for f32 scores, exponentials and sums (scores here stay below 100,
       so an f32 score is off by at most 100 * 2^-17 from 128 f32 additions, and
       in practice by far less)
  lse: dim * 2^-23 * max_p scale * sum_i |q_i k_i| for f32 additions in any order,
       + 1e-5 for the exponentials' sum
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu

dsp = pytest.importorskip("speculative_decoding_draft_02_gb300")

U = 2.0 ** -9


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from speculative_decoding_draft_02_gb300 import build
    build.build()
    dsp.load_library()
    yield
    assert dsp.dspark_device_status() == 0


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def host(t):
    if t.dtype in (torch.bfloat16, torch.float8_e4m3fn):
        t = t.float()
    return t.cpu().numpy()


def random_parents(rng, R, gamma):
    return np.array([[int(rng.integers(max(0, j - 5), j)) for j in range(1, gamma + 1)]
                     for _ in range(R)], dtype=np.int32).reshape(R, gamma)


# -------------------------------------------------------------------- plan ----

def run_plan(ctx, length, extra, parent, ps, held, n_free, free, table, n_rows, alias=False,
             masks=True):
    R = len(ctx)
    held_d, nf_d, free_d, table_d = i32(held), i32([n_free]), i32(free), i32(table)
    held_o, nf_o = (held_d, nf_d) if alias else (torch.full_like(held_d, -9), i32([-9]))
    row_start = i32(np.full(R + 1, -9))
    position = i32(np.full(n_rows, -9))
    slot = torch.full((n_rows,), -9, dtype=torch.int64, device="cuda")
    anc = torch.full((n_rows,), -9, dtype=torch.int64, device="cuda") if masks else None
    dsp.dspark_kv_plan(i32(ctx), i32(length), extra, None if parent is None else i32(parent), ps,
                       held_d, nf_d, free_d, table_d, held_o, nf_o, row_start, position, slot, anc)
    torch.cuda.synchronize()
    out = dict(row_start=row_start, position=position, slot=slot, held=held_o, n_free=nf_o,
               free_pages=free_d, block_table=table_d)
    out = {k: host(v) for k, v in out.items()}
    if masks:
        out["anc"] = host(anc).view(np.uint64)
    return out


def random_pool(rng, R, ps, max_pages, ctx, spare):
    """Pages dealt in random order: (held, n_free, stack, table)."""
    held = np.array([-(-max(c, 0) // ps) for c in ctx])
    ids = rng.permutation(int(held.sum()) + spare)
    table = np.full((R, max_pages), -7, dtype=np.int64)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    free = np.full(len(ids), -3)
    free[:spare] = ids[at:]
    return held, spare, free, table


# R, gamma, tree, extra, page, ctx range, alias
PLANS = [
    (1, 1, False, 1, 16, (0, 1), False),
    (4, 5, False, 1, 16, (0, 40), True),
    (32, 31, True, 1, 16, (0, 300), False),    # one CTA's requests, and one more
    (33, 63, True, 1, 32, (0, 300), True),
    (300, 7, True, 1, 64, (0, 500), False),
    (1025, 3, False, 1, 16, (0, 100), False),
    (2000, 40, True, 1, 128, (0, 100), True),
    (3, 3000, False, 0, 256, (0, 5), False),   # prompts: no masks
]


@pytest.mark.parametrize("R,gamma,tree,extra,ps,span,alias", PLANS)
def test_plan_matches_oracle(R, gamma, tree, extra, ps, span, alias):
    rng = np.random.default_rng(1000 + R + gamma)
    ctx = rng.integers(span[0], span[1] + 1, R)
    length = rng.integers(0, gamma + 1, R)
    max_pages = -(-(span[1] + gamma + 1) // ps) + 1
    held, n_free, free, table = random_pool(rng, R, ps, max_pages, ctx, R * (gamma // ps + 2))
    if R > 2:
        ctx[rng.random(R) < 0.2] = -1
    parent = random_parents(rng, R, gamma) if tree else None
    n_rows = R * (gamma + 1) + 5
    masks = gamma < 64
    got = run_plan(ctx, length, extra, parent, ps, held, n_free, free, table, n_rows, alias, masks)
    want = oc.kv_plan(ctx, length, extra, parent, ps, held, n_free, free, table, n_rows)
    for name, x in got.items():
        np.testing.assert_array_equal(x.reshape(-1), np.asarray(want[name]).reshape(-1), name)
    assert dsp.dspark_device_status() == 0


def test_plan_starved_of_pages():
    rng = np.random.default_rng(5)
    R, ps = 40, 16
    ctx = rng.integers(0, 60, R)
    length = rng.integers(0, 30, R)
    held, n_free, free, table = random_pool(rng, R, ps, 6, ctx, 11)
    got = run_plan(ctx, length, 1, None, ps, held, n_free, free, table, 40 * 31)
    want = oc.kv_plan(ctx, length, 1, None, ps, held, n_free, free, table, 40 * 31)
    for name, x in got.items():
        np.testing.assert_array_equal(x.reshape(-1), np.asarray(want[name]).reshape(-1), name)
    assert dsp.dspark_device_status() == 9


def test_plan_reports_bad_inputs_on_the_device():
    base = dict(extra=1, parent=None, ps=16, held=[1], n_free=2, free=[1, 2, 0, 0],
                table=[[3, -7]], n_rows=8)

    def status(ctx, length, **kw):
        a = {**base, **kw}
        out = run_plan([ctx], [length], a["extra"], a["parent"], a["ps"], a["held"], a["n_free"],
                       a["free"], a["table"], a["n_rows"])
        return dsp.dspark_device_status(), out

    assert status(3, 2)[0] == 0
    rc, out = status(3, -1)                       # a negative length gives no rows
    assert rc == 6 and out["row_start"].tolist() == [0, 0] and (out["slot"] == -1).all()
    assert status(3, 9)[0] == 6                   # ten rows in a buffer of eight
    rc, out = status(30, 5)                       # longer than its two pages
    assert rc == 6 and (out["slot"][2:] == -1).all() and out["n_free"].tolist() == [2]
    assert status(3, 2, held=[5])[0] == 9
    assert status(3, 2, n_free=77)[0] == 9
    rc, out = status(3, 2, parent=[[0, 2]])       # a node cannot be its own parent
    assert rc == 3 - 2 and out["anc"].tolist()[:3] == [1, 3, 5]


# ------------------------------------------------------------------ append ----

def make_cache(n_pages, ps, heads, dim, fp8, order="token", fill=None, scales=True, seed=0):
    """A cache filled with random values (or `fill`): [n_pages, ps, heads, dim] views of a
    token-major, head-major or padded buffer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def one():
        shape = dict(token=(n_pages, ps, heads, dim), head=(n_pages, heads, ps, dim),
                     padded=(n_pages, ps, heads + 1, 2 * dim))[order]
        t = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        if fill is not None:
            t.fill_(fill)
        t = t.to(torch.float8_e4m3fn) if fp8 else t
        if order == "head":
            return t.permute(0, 2, 1, 3)
        return t[:, :, :heads, dim:] if order == "padded" else t

    k, v = one(), one()
    ks = vs = None
    if fp8 and scales:
        ks, vs = (0.25 + torch.rand(heads, generator=g, device="cuda") for _ in range(2))
    return dsp.KVCache(k, v, ks, vs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,heads,dim,ps,order,fused", [
    (1, 1, 64, 16, "token", False),
    (37, 3, 128, 32, "head", True),
    (700, 8, 128, 64, "padded", True),
    (513, 5, 64, 256, "token", True),
])
def test_append_matches_oracle(rows, heads, dim, ps, order, fused, fp8):
    rng = np.random.default_rng(rows)
    n_pages = -(-rows // ps) + 3
    cache = make_cache(n_pages, ps, heads, dim, fp8, order, seed=rows)
    slot = rng.permutation(n_pages * ps)[:rows]
    slot[rng.random(rows) < 0.2] = -1
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + 1)
    both = 30 * torch.randn((rows, 2 * heads, dim), generator=g, device="cuda")
    both[0, :, :4] = torch.tensor([math.inf, -math.inf, 1e6, 1e-6])
    both[-1, :, 5] = math.nan
    both = both.to(torch.bfloat16)
    k, v = both[:, :heads], both[:, heads:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    want = [oc.kv_append(host(c), host(x), slot, None if s is None else host(s))
            for c, x, s in ((cache.k, k, cache.k_scale), (cache.v, v, cache.v_scale))]
    dsp.dspark_kv_append(cache, k, v, torch.tensor(slot, device="cuda"))
    np.testing.assert_array_equal(host(cache.k), want[0])
    np.testing.assert_array_equal(host(cache.v), want[1])


def test_append_slots_outside_the_cache():
    cache = make_cache(2, 16, 2, 64, False, seed=3)
    before = host(cache.k)
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    dsp.dspark_kv_append(cache, x, x, torch.tensor([32, -5, 1 << 40], device="cuda"))
    assert dsp.dspark_device_status() == 9
    np.testing.assert_array_equal(host(cache.k), before)
    dsp.dspark_kv_append(cache, x[:0], x[:0], torch.empty(0, dtype=torch.int64, device="cuda"))


# --------------------------------------------------------------- attention ----

def attention_case(ctx, ns, heads_q, heads, dim, ps, fp8=False, order="token", tree=True, seed=0,
                   anc=None, spare=2, q_std=2.0, poison=True):
    """A batch in its pages, everything past each request's tokens NaN."""
    rng = np.random.default_rng(seed)
    R = len(ctx)
    pages = [-(-(c + n) // ps) for c, n in zip(ctx, ns)]
    max_pages = max(pages) + 1
    n_pages = sum(pages) + spare
    cache = make_cache(n_pages, ps, heads, dim, fp8, order, seed=seed)
    ids = rng.permutation(n_pages)
    table = np.full((R, max_pages), -1)
    at = 0
    if poison:
        used = torch.zeros((n_pages, ps), dtype=torch.bool)
    for r in range(R):
        table[r, :pages[r]] = ids[at:at + pages[r]]
        at += pages[r]
        if poison:
            for p in range(ctx[r] + ns[r]):
                used[table[r, p // ps], p % ps] = True
    if poison:
        bad = ~used.cuda()
        for t in (cache.k, cache.v):
            f = t.float()
            f[bad] = math.nan
            t.copy_(f.to(t.dtype))
    row_start = np.concatenate([[0], np.cumsum(ns)])
    rows = int(row_start[-1]) + 3
    if anc is None and tree:
        words = []
        for n in ns:
            parent = random_parents(rng, 1, max(n - 1, 1))[0]
            words += [sum(1 << j for j in s) for s in oc.ancestors(parent, n)]
        anc = np.array(words + [0] * 3, dtype=np.uint64)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7)
    wide = torch.randn((rows, heads_q + 2, dim), generator=g, device="cuda") * q_std
    return dict(cache=cache, ctx=np.array(ctx), ns=ns, row_start=row_start, anc=anc, table=table,
                q=wide.to(torch.bfloat16)[:, 1:1 + heads_q], scale=1 / math.sqrt(dim), rows=rows)


def run_attention(c, max_nodes=None, stream=None, ws=None, want_lse=True):
    cache, q = c["cache"], c["q"]
    rows, heads_q, dim = q.shape
    out = torch.full((rows, heads_q + 1, dim), -77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, heads_q), -77.0, device="cuda") if want_lse else None
    max_nodes = max_nodes or max(max(c["ns"]), 1)
    R = len(c["ctx"])
    if ws is None:
        ws = dsp.workspace(dsp.dspark_tree_attention_workspace_bytes(cache, R, heads_q, max_nodes))
        ws.fill_(255)  # contents on entry are ignored: NaN patterns
    anc = None if c["anc"] is None else torch.tensor(c["anc"].view(np.int64), device="cuda")
    args = (cache, q, i32(c["ctx"]), i32(c["row_start"]), anc, i32(c["table"]), max_nodes,
            c["scale"], out[:, :heads_q], lse, ws)
    torch.cuda.synchronize()
    dsp.dspark_tree_attention(*args, stream=stream)
    torch.cuda.synchronize()
    assert (out[:, heads_q] == -77).all()
    return out[:, :heads_q], lse


def check_attention(c, out, lse, rows=None):
    cache = c["cache"]
    q, k, v = (np.float64(host(t)) for t in (c["q"], cache.k, cache.v))
    ks, vs = (None if s is None else np.float64(host(s)) for s in (cache.k_scale, cache.v_scale))
    args = (c["ctx"], c["row_start"], c["anc"], c["table"], c["scale"])
    want, want_lse = oc.tree_attention(q, k, v, *args, ks, vs)
    size, _ = oc.tree_attention(q, k, np.abs(v), *args, ks, vs)
    top = np.nanmax(np.abs(np.where(np.isfinite(k), k, 0))) * (1 if ks is None else ks.max())
    total = int(c["row_start"][-1])
    got, got_lse = np.float64(host(out)), np.float64(host(lse))
    assert (got[total:] == -77).all() and (got_lse[total:] == -77).all()
    pick = slice(0, total) if rows is None else rows
    got, want, size = got[pick], want[pick], size[pick]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    err = np.abs(got - want)
    tol = U * np.abs(want) + (U + 2e-4) * size + 1e-30
    assert (np.isnan(want) | (err <= tol)).all(), np.nanmax(err / tol)
    bound = (q.shape[2] * 2.0 ** -23 * c["scale"] * np.abs(q).sum(-1)[pick] * top + 1e-5)
    a, b = got_lse[pick], want_lse[pick]
    fine = np.isfinite(b)
    np.testing.assert_array_equal(a[~fine], b[~fine])
    assert (np.abs(a - b)[fine] <= bound[fine]).all(), np.max(np.abs(a - b)[fine] / bound[fine])


EDGES = [0, 1, 15, 16, 17, 127, 128, 129, 255, 300]

# ctx, rows, heads_q, heads, dim, page, options
ATTENTION = {
    "self_only": ([0], [1], 4, 4, 64, 16, {}),
    "single_token": ([1000], [1], 32, 8, 128, 16, {}),
    "one_row_each": (EDGES, [1] * 10, 8, 2, 128, 32, dict(tree=False)),
    "ragged_trees": (EDGES, [1, 0, 7, 64, 33, 5, 64, 2, 17, 31], 10, 2, 64, 16, {}),
    "ragged_trees_128": (EDGES, [9, 1, 64, 0, 2, 12, 64, 40, 6, 1], 8, 2, 128, 64, {}),
    "chains_by_default": ([5, 130, 250], [6, 9, 64], 6, 3, 128, 128, dict(tree=False)),
    "multi_query": ([70, 3], [64, 50], 16, 1, 128, 32, {}),
    "multi_head": ([300, 40], [6, 1], 7, 7, 64, 256, dict(order="head")),
    "group_of_64": ([40, 129], [2, 1], 64, 1, 64, 16, dict(order="padded")),
    "group_of_33": ([90], [5], 66, 2, 128, 16, {}),
    "page_256": ([511, 513], [3, 4], 12, 4, 128, 256, dict(order="padded")),
    "long": ([20000, 9], [5, 3], 8, 1, 128, 64, {}),
    "long_64": ([9001], [1], 3, 1, 64, 16, {}),
    "peaked": ([700], [16], 8, 2, 128, 16, dict(q_std=12.0)),
    "many": ([int(x) for x in np.random.default_rng(1).integers(0, 60, 200)],
             [int(x) for x in np.random.default_rng(2).integers(0, 5, 200)], 4, 2, 64, 16, {}),
}


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(ATTENTION))
def test_attention_matches_oracle(name, fp8):
    ctx, ns, heads_q, heads, dim, ps, kw = ATTENTION[name]
    kw = dict(kw)
    if fp8 and "q_std" in kw:
        kw["q_std"] /= 2
    c = attention_case(ctx, ns, heads_q, heads, dim, ps, fp8=fp8, seed=len(name), **kw)
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    again, lse2 = run_attention(c)   # the same bits from call to call
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_attention_rows_that_see_nothing(fp8):
    # row 1 of request 0 sees nothing; request 1's rows see only node 2, whose bits past
    # the request's rows are ignored
    anc = np.array([1, 0, 5, 4 | 1 << 40, 1 << 2, 4, 0, 0, 0], dtype=np.uint64)
    c = attention_case([0, 0], [3, 3], 4, 2, 64, 16, fp8=fp8, anc=anc, seed=9)
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_masked_nodes_do_not_reach_other_rows(fp8, dim):
    # nodes 2 and 5 hold NaN (and infinities) in K and V: only rows that see them carry them
    n, ctx = 9, 121
    anc = np.array([1, 3, 5, 9, 19, 37, 64 | 1, 128 | 9, 256 | 64 | 1, 0, 0, 0], dtype=np.uint64)
    c = attention_case([ctx], [n], 6, 2, dim, 16, fp8=fp8, anc=anc, seed=4)
    clean, clean_lse = run_attention(c)
    for node, value in ((2, math.nan), (5, math.nan if fp8 else math.inf)):
        page, at = c["table"][0, (ctx + node) // 16], (ctx + node) % 16
        for t in (c["cache"].k, c["cache"].v):
            row = t[page, at].float()
            row[:, 3:9] = value
            t[page, at] = row.to(t.dtype)
    out, lse = run_attention(c)
    sees = np.array([bool(int(w) & (1 << 2 | 1 << 5)) for w in anc[:n]])
    assert torch.equal(out[:n][~sees], clean[:n][~sees])
    assert torch.equal(lse[:n][~sees], clean_lse[:n][~sees])
    assert torch.isnan(out[:n][sees].float()[:, :, 3:9]).all()
    # V alone: the scores, and every other column of the rows that see it, stay
    c = attention_case([ctx], [n], 6, 2, dim, 16, fp8=fp8, anc=anc, seed=4)
    page, at = c["table"][0, (ctx + 2) // 16], (ctx + 2) % 16
    row = c["cache"].v[page, at].float()
    row[:, 7] = math.nan
    c["cache"].v[page, at] = row.to(c["cache"].v.dtype)
    out, lse = run_attention(c)
    assert torch.equal(lse[:n], clean_lse[:n])
    see2 = torch.tensor([bool(int(w) & 4) for w in anc[:n]])
    assert torch.isnan(out[:n][see2][:, :, 7].float()).all()
    keep = torch.ones(dim, dtype=torch.bool)
    keep[7] = False
    assert torch.equal(out[:n][~see2], clean[:n][~see2])
    np.testing.assert_allclose(host(out[:n])[:, :, keep.numpy()], host(clean[:n])[:, :, keep.numpy()],
                               rtol=4 * U, atol=4 * U)


def test_attention_on_another_stream_and_without_lse():
    c = attention_case([300, 2], [6, 3], 8, 2, 128, 16, seed=21)
    want, _ = run_attention(c)
    s = torch.cuda.Stream()
    got, _ = run_attention(c, stream=s, want_lse=False)
    assert torch.equal(got, want)


def test_attention_offsets_past_32_bits():
    # pages of 8 x 256 x 128 elements; the used ones lie past 2^32 bytes and 2^31 elements
    ps, heads, dim, n_pages = 256, 8, 128, 8400
    k, v = (torch.empty((n_pages, ps, heads, dim), dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    assert k.numel() > 2 ** 31
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    small = [torch.randn((4, ps, heads, dim), generator=g, device="cuda").to(torch.bfloat16)
             for _ in range(2)]
    k[-4:], v[-4:] = small
    ctx, n = 2 * ps + 17, 4
    table = np.array([[n_pages - 2, n_pages - 4, n_pages - 1, 0]])
    c = dict(cache=dsp.KVCache(k, v), ctx=np.array([ctx]), ns=[n], row_start=np.array([0, n]),
             anc=None, table=table, scale=1 / math.sqrt(dim), rows=n,
             q=(2 * torch.randn((n, 8, dim), generator=g, device="cuda")).to(torch.bfloat16))
    # new rows through the same far slots
    rows = torch.randn((n, heads, dim), generator=g, device="cuda").to(torch.bfloat16)
    slot = torch.tensor([(n_pages - 1) * ps + 17 + i for i in range(n)], device="cuda")
    dsp.dspark_kv_append(c["cache"], rows, rows, slot)
    assert torch.equal(k[-1, 17:17 + n], rows) and torch.equal(v[-1, 17:17 + n], rows)
    out, lse = run_attention(c)
    near = dsp.KVCache(k[-4:].clone(), v[-4:].clone())
    c2 = dict(c, cache=near, table=np.array([[2, 0, 3, 0]]))
    out2, lse2 = run_attention(c2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    check_attention(c2, out2, lse2)
    # and a path moved there
    dsp.dspark_kv_compact(c["cache"], i32([ctx]), i32([1]), i32([[3, -1, -1]]), i32(table))
    assert torch.equal(k[-1, 18], rows[3]) and torch.equal(v[-1, 18], rows[3])
    del k, v, c
    torch.cuda.empty_cache()


def test_attention_reports_bad_inputs_on_the_device():
    c = attention_case([40, 20], [6, 3], 8, 2, 128, 16, seed=31, poison=False)
    want, _ = run_attention(c)
    # more rows than max_nodes: the first ones are computed, the rest left as they were
    out, _ = run_attention(c, max_nodes=4)
    assert dsp.dspark_device_status() == 6
    assert torch.equal(out[6:9], want[6:9]) and (out[4:6] == -77).all()
    # a page outside the cache reads as zeros
    table = c["table"].copy()
    c["table"][1, 0] = 10 ** 6
    out, lse = run_attention(c)
    assert dsp.dspark_device_status() == 9
    assert torch.equal(out[:6], want[:6]) and torch.isfinite(out[:9].float()).all()
    # a request longer than its table is cut there
    c["table"] = table[:, :2]
    out, lse = run_attention(c)
    assert dsp.dspark_device_status() == 6 and torch.equal(out[6:9], want[6:9])


# -------------------------------------------------------- accept, compact ----

@pytest.mark.parametrize("R,gamma,tree", [(1, 1, False), (4, 5, True), (33, 32, True),
                                          (300, 63, True), (70, 8, False)])
def test_accept_and_compact_match_oracle(R, gamma, tree):
    rng = np.random.default_rng(R + gamma)
    ns = rng.integers(0, gamma + 2, R)
    if R == 1:
        ns[:] = gamma + 1
    row_start = np.concatenate([[0], np.cumsum(ns)])
    parent = random_parents(rng, R, gamma) if tree else None
    tokens = rng.integers(0, 3, (R, gamma))
    choice = rng.integers(0, 3, row_start[-1] + 2)
    ctx = rng.integers(0, 100, R)
    outs = [i32(np.full(s, -9)) for s in (R, R, (R, gamma), R)]
    dsp.dspark_tree_accept(i32(row_start), None if parent is None else i32(parent), i32(tokens),
                           i32(choice), i32(ctx), *outs)
    acc, bonus, paths, ctx_out = oc.tree_accept(row_start, parent, tokens, choice, ctx)
    np.testing.assert_array_equal(host(outs[0]), acc)
    np.testing.assert_array_equal(host(outs[1]), bonus)
    full = np.full((R, gamma), -1)
    for r, p in enumerate(paths):
        full[r, :len(p)] = p
    np.testing.assert_array_equal(host(outs[2]), full)
    np.testing.assert_array_equal(host(outs[3]), ctx_out)
    same = i32(ctx)  # ctx_out may be ctx
    dsp.dspark_tree_accept(i32(row_start), None if parent is None else i32(parent), i32(tokens),
                           i32(choice), same, *outs[:3], same)
    np.testing.assert_array_equal(host(same), ctx_out)
    # the paths' K and V
    ps = 16
    pages = [-(-(c + gamma + 1) // ps) for c in ctx]
    table = np.full((R, max(pages)), -1)
    ids = rng.permutation(sum(pages))
    for r in range(R):
        table[r, :pages[r]], ids = ids[:pages[r]], ids[pages[r]:]
    for heads, dim, fp8, order in ((2, 64, False, "token"), (3, 128, True, "head"),
                                   (5, 128, False, "padded")):
        cache = make_cache(sum(pages), ps, heads, dim, fp8, order, seed=R)
        want = [oc.kv_compact(host(t), ctx, paths, table) for t in (cache.k, cache.v)]
        dsp.dspark_kv_compact(cache, i32(ctx), outs[0], outs[2], i32(table))
        np.testing.assert_array_equal(host(cache.k), want[0])
        np.testing.assert_array_equal(host(cache.v), want[1])


def test_accept_and_compact_report_bad_inputs_on_the_device():
    outs = [i32(np.full(s, -9)) for s in (1, 1, (1, 3), 1)]
    row, tok = i32([0, 4]), i32([[1, 1, 1]])
    dsp.dspark_tree_accept(row, i32([[0, 2, 1]]), tok, i32([1, 1, 1, 1]), i32([5]), *outs)
    assert dsp.dspark_device_status() == 1
    assert host(outs[2]).tolist() == [[1, 3, -1]]        # node 2 has no parent before it
    dsp.dspark_tree_accept(i32([0, 9]), None, tok, i32([1, 1, 1, 1]), i32([5]), *outs)
    assert dsp.dspark_device_status() == 6 and host(outs[1]).tolist() == [-1]
    cache = make_cache(2, 16, 2, 64, False, seed=3)
    before = host(cache.k)
    for path, table, rc in (([[2, 2, -1]], [[0, 1]], 1), ([[64, 1, -1]], [[0, 1]], 1),
                            ([[2, 3, -1]], [[-1, 1]], 9), ([[2, 3, -1]], [[2, 1]], 9)):
        dsp.dspark_kv_compact(cache, i32([4]), i32([2]), i32(path), i32(table))
        assert dsp.dspark_device_status() == rc
        np.testing.assert_array_equal(host(cache.k), before)


# ---------------------------------------------------------------- refusals ----

def test_binding_refuses_wrong_tensors():
    c = attention_case([40], [3], 8, 2, 128, 16, seed=1, poison=False)
    cache, q = c["cache"], c["q"]
    ws = dsp.workspace(dsp.dspark_tree_attention_workspace_bytes(cache, 1, 8, 3))
    out = torch.empty_like(q)
    good = dict(q=q, ctx=i32(c["ctx"]), row_start=i32(c["row_start"]),
                anc=torch.tensor(c["anc"].view(np.int64), device="cuda"), table=i32(c["table"]),
                out=out, ws=ws, nodes=3)

    def call(**kw):
        a = {**good, **kw}
        dsp.dspark_tree_attention(cache, a["q"], a["ctx"], a["row_start"], a["anc"], a["table"],
                                  a["nodes"], 0.1, a["out"], None, a["ws"])

    call()
    for kw in (dict(q=q.float()), dict(q=q[:, :, ::2]), dict(q=q[:, :7]), dict(q=q[1:]),
               dict(ctx=good["ctx"].long()), dict(row_start=good["row_start"][:1]),
               dict(anc=good["anc"][:2]), dict(table=good["table"][0]), dict(nodes=0),
               dict(nodes=65), dict(ws=ws[:16]), dict(ws=ws.cpu()), dict(out=out.cpu()),
               dict(q=torch.randn((6, 9, 131), device="cuda").bfloat16()[:, 1:, 1:129])):
        with pytest.raises(dsp.DSparkError):
            call(**kw)
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in ((x[:1], x, slot), (x, x, slot.int()), (x.half(), x.half(), slot),
                (x, x.transpose(0, 1).contiguous().transpose(0, 1), slot)):
        with pytest.raises(dsp.DSparkError):
            dsp.dspark_kv_append(cache, *bad)
    k = torch.zeros((2, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    for args in ((k, k[:1]), (k, k.half()), (k.half(), k.half()), (k[0], k[0]),
                 (k.cpu(), k.cpu()), (k, k, torch.ones(2, device="cuda"))):
        with pytest.raises(dsp.DSparkError):
            dsp.KVCache(*args)
    with pytest.raises(dsp.DSparkError):
        dsp.dspark_kv_plan(i32([1]), i32([1]), 1, None, 24, i32([1]), i32([0]), i32([0]),
                           i32([[0]]), i32([1]), i32([0]), i32([0, 0]), i32([0, 0]),
                           torch.zeros(2, dtype=torch.int64, device="cuda"))


def test_entry_points_refuse_bad_arguments():
    lib = dsp.load_library()
    fake = ctypes.c_void_p(4096)

    def cache(**kw):
        f = dict(k=4096, v=8192, k_scale=None, v_scale=None, page_stride=16 * 2 * 64,
                 token_stride=128, head_stride=64, n_pages=4, page_size=16, heads=2, dim=64,
                 type=0)
        return ctypes.byref(dsp.KVCacheStruct(**{**f, **kw}))

    size = lib.dspark_tree_attention_workspace_bytes
    assert size(cache(), 4, 8, 6) > 0
    bad = [dict(k=None), dict(v=4104), dict(dim=96), dict(heads=0), dict(page_size=48),
           dict(page_size=8), dict(page_size=512), dict(n_pages=0), dict(type=2),
           dict(token_stride=60), dict(head_stride=0), dict(page_stride=1 << 41),
           dict(type=1, head_stride=72)]
    for kw in bad:
        assert size(cache(**kw), 4, 8, 6) == 0, kw
        assert lib.dspark_kv_append(cache(**kw), 1, fake, fake, 128, 64, fake, None) == 1
        assert lib.dspark_kv_compact(cache(**kw), 1, 5, 2, fake, fake, fake, fake, None) == 1
    for R, hq, nodes in ((0, 8, 6), (4, 7, 6), (4, 8, 0), (4, 8, 65), (4, 2 * 65, 6)):
        assert size(cache(), R, hq, nodes) == 0

    def attn(c=None, R=4, hq=8, nodes=6, rows=24, pages=3, q=fake, q_row=512, q_head=64,
             table=fake, out=fake, ws=fake, nbytes=1 << 40):
        return lib.dspark_tree_attention(c or cache(), R, hq, nodes, rows, pages, q, q_row, q_head,
                                         fake, fake, None, table, 0.1, out, 512, 64, None, ws,
                                         nbytes, None)

    for kw in (dict(q=None), dict(q_row=4), dict(q_head=0), dict(q=ctypes.c_void_p(4098)),
               dict(table=None), dict(out=None), dict(out=ctypes.c_void_p(4097)), dict(pages=0),
               dict(rows=-1), dict(hq=9)):
        assert attn(**kw) == 1, kw
    assert attn(ws=None) == 4 and attn(nbytes=16) == 4 and attn(ws=ctypes.c_void_p(4224)) == 4
    assert lib.dspark_kv_append(cache(), 1, None, fake, 128, 64, fake, None) == 1
    assert lib.dspark_kv_append(cache(), 1, fake, fake, 124, 64, fake, None) == 1
    assert lib.dspark_tree_accept(1, 64, 1, *[fake] * 9, None) == 1
    assert lib.dspark_tree_accept(1, 5, 1, None, *[fake] * 8, None) == 1
    assert lib.dspark_kv_compact(cache(), 70000, 5, 2, fake, fake, fake, fake, None) == 8
    plan = lambda R, gamma, extra, ps, parent=fake, ctx=fake: lib.dspark_kv_plan(  # noqa: E731
        R, gamma, extra, 10, ps, 4, 2, ctx, fake, parent, *[fake] * 10, None)
    assert plan(0, 5, 1, 16) == 1 and plan(1, 64, 1, 16) == 1 and plan(1, 5, 0, 16) == 1
    assert plan(1, 5, 2, 16, None) == 1 and plan(1, 5, 1, 24) == 1
    assert plan(1, 5, 1, 16, ctx=None) == 1 and plan(20000, 5, 1, 16) == 8
