"""Attention of drafted token trees on the GPU against the float64 oracle.

Tolerances are those of the other attention tests (``gpu_support``): fp32
1e-5, fp16 / bf16 max(2e-3, 1 ulp).  The kernels hold scores, softmax
statistics and sums in fp32 and enter probabilities with at least 16
significant bits, so beside the output's rounding (half an ulp) there remain
errors of a few 2^-16 of the largest value, far below either bound."""
import math

import pytest
import torch

import oracle
import paged_kv_decode_tables_gb300 as pkv
import workloads
from gpu_support import assert_attention_close, on_device

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from paged_kv_decode_tables_gb300 import _build
    _build.build()


def _tree_mask(drafts, cols, seed):
    """Random ancestor masks, [sum(drafts), cols] bool."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for T in drafts:
        m = torch.zeros(T, cols, dtype=torch.bool)
        for i in range(T):
            parent = i - 1 - int(torch.randint(0, 4, (1,), generator=g))
            if parent >= 0:
                m[i] = m[parent]
            m[i, i] = True
        rows.append(m)
    return torch.cat(rows) if rows else torch.zeros(0, cols, dtype=torch.bool)


def _batch(dtype, kv, D, bs, H, Hk, lens, drafts, seed, mask="tree", alibi=False, **kw):
    inp = workloads.make_inputs(num_heads=H, num_kv_heads=Hk, head_size=D, block_size=bs, dtype=dtype,
                                seq_lens=lens, seed=seed, kv_cache_dtype=kv, k_scale=0.75, v_scale=1.5,
                                alibi=alibi, **kw)
    n = sum(drafts)
    g = torch.Generator().manual_seed(seed + 100)
    inp["query"] = torch.randn(n, H, D, generator=g).to(DT[dtype])
    inp["cu"] = torch.tensor([0] + list(drafts)).cumsum(0).int()
    inp["mask"] = inp["positions"] = None
    if mask == "tree":
        inp["mask"] = _tree_mask(drafts, max(drafts), seed)
        ctx = torch.cat([torch.full((T,), L - T) for L, T in zip(lens, drafts)])
        inp["positions"] = (ctx + inp["mask"].sum(1) - 1).int()
    return inp


def _kwargs(g, cap=0.0):
    return dict(tree_mask=g["mask"], positions=g["positions"], logits_soft_cap=cap,
                kv_cache_dtype=g["kv_cache_dtype"], k_scale=g["k_scale"], v_scale=g["v_scale"],
                alibi_slopes=g["alibi_slopes"])


def _workspace(D):
    """A workspace full of NaN: nothing in it may be read before it is written."""
    n = pkv.tree_workspace_bytes(D)
    return torch.full((n // 4,), math.nan, dtype=torch.float32, device="cuda")


def _run(inp, cap=0.0, err=None, out=None, workspace=None, **over):
    g = on_device(inp)
    out = torch.empty_like(g["query"]) if out is None else out
    pkv.paged_attention_tree(out, g["query"], g["key_cache"], g["value_cache"],
                             over.pop("block_tables", g["block_tables"]), g["seq_lens"], g["cu"],
                             g["scale"], workspace=_workspace(g["head_size"]) if workspace is None else workspace,
                             err_flag=err, **{**_kwargs(g, cap), **over})
    return out


def _oracle(inp, cap=0.0):
    kw = _kwargs(inp, cap)
    if kw["alibi_slopes"] is not None:
        kw["alibi_slopes"] = kw["alibi_slopes"].tolist()
    return oracle.tree_attention(inp["query"], inp["key_cache"], inp["value_cache"], inp["block_tables"],
                                 inp["seq_lens_list"], inp["cu"], inp["scale"], **kw)


CASES = [
    # dtype, kv_cache_dtype, D, bs, H, Hk
    ("bf16", "auto", 128, 16, 32, 8),
    ("bf16", "auto", 64, 8, 4, 4),
    ("bf16", "auto", 128, 32, 14, 2),
    ("bf16", "auto", 256, 16, 8, 1),
    ("bf16", "auto", 256, 32, 4, 4),
    ("f16", "auto", 128, 8, 12, 4),
    ("f16", "auto", 64, 32, 16, 1),
    ("f16", "auto", 64, 16, 6, 2),
    ("f16", "auto", 256, 8, 2, 2),
    ("f32", "auto", 64, 8, 8, 4),
    ("f32", "auto", 128, 16, 8, 2),
    ("f32", "auto", 128, 32, 3, 3),
    ("bf16", "fp8_e4m3", 128, 16, 32, 8),
    ("bf16", "fp8_e5m2", 64, 8, 8, 2),
    ("bf16", "fp8_e5m2", 256, 16, 8, 2),
    ("f16", "fp8_e4m3", 256, 32, 4, 1),
    ("f16", "fp8_e5m2", 128, 32, 6, 3),
    ("f16", "fp8_e4m3", 64, 16, 16, 2),
    ("f16", "fp8", 128, 8, 8, 8),
    ("bf16", "fp8_e4m3", 256, 8, 4, 2),
    ("bf16", "fp8_e4m3", 64, 32, 4, 1),
]


@pytest.mark.parametrize("dtype,kv,D,bs,H,Hk", CASES)
def test_ragged_trees(dtype, kv, D, bs, H, Hk):
    """One token, whole-tree sequences without context, tiles and pages that end
    anywhere, a sequence without drafted tokens, a long one."""
    lens = [1, 7, bs, 130, 3 * bs + 1, 257, 40, 900, 128]
    drafts = [1, 7, 3, 12, 5, 9, 0, 6, 17]
    inp = _batch(dtype, kv, D, bs, H, Hk, lens, drafts, D + bs + H, unused_slot_fill=math.nan)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(inp, err=err)
    assert_attention_close(got, _oracle(inp), DT[dtype], f"{dtype}/{kv} D{D} bs{bs} {H}/{Hk}")
    assert int(err) == 0


@pytest.mark.parametrize("dtype,kv,D,bs,H,Hk", [CASES[i] for i in (0, 5, 10, 12, 3)])
@pytest.mark.parametrize("cap,alibi", [(5.0, False), (50.0, False), (0.0, True), (30.0, True)])
def test_soft_cap_and_alibi(dtype, kv, D, bs, H, Hk, cap, alibi):
    lens, drafts = [400, 33, 9, 150], [5, 16, 9, 1]
    inp = _batch(dtype, kv, D, bs, H, Hk, lens, drafts, 3, alibi=alibi, peaky_fraction=0.02)
    assert_attention_close(_run(inp, cap), _oracle(inp, cap), DT[dtype], f"cap {cap} alibi {alibi}")


@pytest.mark.parametrize("dtype,kv,D,bs,H,Hk", [CASES[i] for i in (0, 10, 12)])
def test_chain_without_a_mask(dtype, kv, D, bs, H, Hk):
    lens, drafts = [300, 20, 64, 5], [8, 20, 1, 2]
    inp = _batch(dtype, kv, D, bs, H, Hk, lens, drafts, 4, mask=None, alibi=True)
    assert_attention_close(_run(inp), _oracle(inp), DT[dtype], "chain")


@pytest.mark.parametrize("dtype,kv,D,H,Hk,T", [
    ("bf16", "auto", 128, 8, 1, 70), ("f16", "fp8_e4m3", 64, 16, 1, 40), ("f32", "auto", 64, 4, 1, 50),
    ("bf16", "auto", 256, 3, 1, 129), ("bf16", "auto", 64, 2, 2, 200)])
def test_many_rows(dtype, kv, D, H, Hk, T):
    """More query rows a kv head than one row tile, whole and cut between CTAs."""
    lens, drafts = [T + 500, T, T + 1], [T, T, T - 3]
    inp = _batch(dtype, kv, D, 16, H, Hk, lens, drafts, 6)
    assert_attention_close(_run(inp), _oracle(inp), DT[dtype], "rows")


@pytest.mark.parametrize("dtype,kv", [("bf16", "auto"), ("f32", "auto"), ("bf16", "fp8_e4m3")])
def test_long_sequence_split_over_the_gpu(dtype, kv):
    """One kv head: every CTA gets a piece of the same unit."""
    inp = _batch(dtype, kv, 128, 16, 4, 1, [30011, 5], [3, 5], 7, peaky_fraction=0.01)
    assert_attention_close(_run(inp), _oracle(inp), DT[dtype], "split")


@pytest.mark.parametrize("dtype,kv,D,bs", [
    ("bf16", "auto", 128, 16), ("bf16", "auto", 128, 32), ("f16", "auto", 64, 8), ("bf16", "auto", 256, 32),
    ("bf16", "fp8_e4m3", 128, 16), ("f16", "fp8_e5m2", 64, 32), ("bf16", "fp8_e5m2", 256, 8), ("f32", "auto", 64, 16)])
def test_many_tiles_to_a_cta(dtype, kv, D, bs):
    """Every CTA goes many times round its ring of tiles, across units."""
    inp = _batch(dtype, kv, D, bs, 8, 8, [6011, 37, 4999, 7001], [2, 5, 3, 1], 19, peaky_fraction=0.01)
    assert_attention_close(_run(inp), _oracle(inp), DT[dtype], "tiles")


@pytest.mark.parametrize("dtype,kv", [("bf16", "auto"), ("f32", "auto"), ("f16", "fp8_e5m2")])
def test_many_short_sequences(dtype, kv):
    """More units than CTAs, several sequences to a CTA; empty ones between."""
    drafts = [(i * 7) % 5 for i in range(700)]
    lens = [t + (i * 13) % 40 for i, t in enumerate(drafts)]
    inp = _batch(dtype, kv, 64, 8, 4, 2, lens, drafts, 8)
    assert_attention_close(_run(inp), _oracle(inp), DT[dtype], "short")


@pytest.mark.parametrize("dtype,kv", [("bf16", "auto"), ("f32", "auto"), ("f16", "fp8_e4m3")])
def test_rows_that_see_nothing(dtype, kv):
    """Without context, a row whose mask is empty gives zeros; one that sees a single token, its value."""
    lens, drafts = [6, 40], [6, 40]
    inp = _batch(dtype, kv, 128, 16, 4, 2, lens, drafts, 9)
    inp["mask"][2] = False
    inp["mask"][6:40] = False
    got = _run(inp)
    assert bool((got[2] == 0).all()) and bool((got[6:40] == 0).all())
    assert_attention_close(got, _oracle(inp), DT[dtype], "empty rows")
    inp["mask"] = torch.zeros(46, 0, dtype=torch.bool)  # no columns: nothing drafted is seen
    assert bool((_run(inp) == 0).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,kv,D", [("bf16", "auto", 128), ("f16", "auto", 64), ("f32", "auto", 128),
                                       ("bf16", "fp8_e5m2", 128), ("bf16", "auto", 256)])
def test_unseen_tokens_may_hold_anything(dtype, kv, D, bad):
    """A drafted token whose key and value are not finite reaches only the rows that see it."""
    lens, drafts = [140, 10], [12, 10]
    inp = _batch(dtype, kv, D, 16, 4, 2, lens, drafts, 10)
    for s, j in ((0, 3), (1, 0)):
        t = lens[s] - drafts[s] + j
        blk, off = int(inp["block_tables"][s, t // 16]), t % 16
        if kv == "auto":
            inp["key_cache"][blk, :, :, off], inp["value_cache"][blk, :, :, off] = bad, bad
        else:
            code = torch.tensor([bad]).to(torch.float8_e5m2).view(torch.uint8)[0]
            inp["key_cache"][blk, :, :, off], inp["value_cache"][blk, :, :, off] = code, code
    got, ref = _run(inp).cpu(), _oracle(inp)
    seen = torch.cat([inp["mask"][:12, 3], inp["mask"][12:, 0]])
    assert bool(seen.any()) and not bool(seen.all())
    assert bool(torch.isfinite(got[~seen].float()).all())
    assert_attention_close(got[~seen], ref[~seen], DT[dtype], "unseen")
    assert bool(torch.isnan(got[seen].float()).all())  # a score that is NaN, or inf - inf


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 256), ("f32", 64)])
def test_a_seen_value_that_is_not_finite_stays(dtype, D):
    """Only the value: its dim is not finite in the rows that see the token, nowhere else."""
    inp = _batch(dtype, "auto", D, 16, 4, 2, [140], [12], 10)
    blk, off = int(inp["block_tables"][0, 131 // 16]), 131 % 16
    inp["value_cache"][blk, 0, 5, off] = math.inf
    inp["value_cache"][blk, 0, D - 3, off] = math.nan
    inp["value_cache"][blk, 1, 0, off] = -math.inf
    got, ref = _run(inp).cpu().double(), _oracle(inp)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(torch.isinf(got), torch.isinf(ref)) and torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
    ok = torch.isfinite(ref)
    assert_attention_close(torch.where(ok, got, 0.0), torch.where(ok, ref, 0.0), DT[dtype], "finite part")


def test_strides_and_page_lists():
    """Query and output with gaps, a mask of bytes with strides, a shared mask row, the flat page list."""
    lens, drafts = [150, 31, 8], [6, 9, 8]
    inp = _batch("bf16", "auto", 128, 16, 8, 2, lens, drafts, 11, bt_col_step=2)
    ref = _oracle(inp)
    g = on_device(inp)
    n = 23
    wide = torch.zeros(n, 11, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = g["query"]
    res = torch.full((n + 4, 9, 130), 7.0, dtype=torch.bfloat16, device="cuda")
    mask = torch.zeros(g["mask"].shape[1], 2 * n, dtype=torch.uint8, device="cuda")
    mask[:, ::2] = g["mask"].t()
    table = inp["block_tables_storage"].cuda()[:, ::2]
    pkv.paged_attention_tree(res[:n, :8, 1:129], wide[:, 2:10], g["key_cache"], g["value_cache"], table,
                             g["seq_lens"], g["cu"], g["scale"], workspace=_workspace(128),
                             tree_mask=mask[:, ::2].t())
    assert_attention_close(res[:n, :8, 1:129], ref, torch.bfloat16, "strides")
    assert bool((res[n:] == 7).all()) and bool((res[:, 8:] == 7).all()) and bool((res[..., 0] == 7).all())
    pages = torch.tensor(sum(inp["block_rows"], []), dtype=torch.int32).cuda()
    indptr = torch.tensor([0] + [len(r) for r in inp["block_rows"]]).cumsum(0).int().cuda()
    assert torch.equal(_run(inp, block_tables=pages, kv_indptr=indptr), _run(inp))
    # inner stride 2
    q2 = torch.zeros(n, 8, 256, dtype=torch.bfloat16, device="cuda")
    q2[..., ::2] = g["query"]
    o2 = torch.zeros_like(q2)
    pkv.paged_attention_tree(o2[..., ::2], q2[..., ::2], g["key_cache"], g["value_cache"], table, g["seq_lens"],
                             g["cu"], g["scale"], workspace=_workspace(128), tree_mask=g["mask"])
    assert torch.equal(o2[..., ::2], _run(inp)) and bool((o2[..., 1::2] == 0).all())
    # one mask row for all: stride 0
    one = torch.tensor([[1, 0, 1, 1]], dtype=torch.uint8)
    inp["mask"] = one.expand(n, 4)
    got = _run(inp, tree_mask=one.cuda().expand(n, 4))
    assert_attention_close(got, _oracle(inp), torch.bfloat16, "shared row")


def test_rows_behind_the_last_sequence():
    """A padded batch: sequences without drafted tokens, rows that belong to none."""
    inp = _batch("bf16", "auto", 128, 16, 8, 2, [100, 0, 0], [4, 0, 0], 12, mask=None)
    inp["query"] = torch.cat([inp["query"], torch.full((5, 8, 128), math.nan).bfloat16()])
    out = torch.full((9, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    _run(inp, out=out)
    assert_attention_close(out[:4], _oracle(inp)[:4], torch.bfloat16, "rows")
    assert bool((out[4:] == 3).all())


@pytest.mark.parametrize("dtype,kv", [("bf16", "auto"), ("f32", "auto")])
def test_bad_device_data_is_flagged(dtype, kv):
    inp = _batch(dtype, kv, 64, 16, 4, 2, [100, 50], [4, 3], 13)

    def err_of(**changes):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = _run({**inp, **changes}, err=err)
        torch.cuda.synchronize()
        return out, int(err)

    good, e = err_of()
    assert e == 0
    bad = inp["block_tables"].clone()
    bad[0, 2] = inp["num_blocks"]
    out, e = err_of(block_tables=bad)
    assert e == pkv.PKV_ERRF_BLOCK_ID and torch.equal(out[4:], good[4:])
    out, e = err_of(seq_lens=torch.tensor([100, 5000], dtype=torch.int32))
    assert e == pkv.PKV_ERRF_SEQ_LEN | (e & pkv.PKV_ERRF_BLOCK_ID) and torch.equal(out[:4], good[:4])
    out, e = err_of(seq_lens=torch.tensor([100, 2], dtype=torch.int32))
    assert e == pkv.PKV_ERRF_SEQ_LEN and torch.equal(out[:4], good[:4])
    out, e = err_of(cu=torch.tensor([0, 4, 9], dtype=torch.int32))
    assert e == pkv.PKV_ERRF_INDPTR and torch.equal(out[:4], good[:4])
    out, e = err_of(cu=torch.tensor([0, -4, 7], dtype=torch.int32))
    assert e == pkv.PKV_ERRF_INDPTR
    out, e = err_of(cu=torch.tensor([5, 4, 7], dtype=torch.int32))
    assert e == pkv.PKV_ERRF_INDPTR and torch.equal(out[4:], good[4:])


@pytest.mark.parametrize("dtype,kv", [("bf16", "auto"), ("bf16", "fp8_e4m3"), ("f32", "auto")])
def test_no_drafted_tokens_at_all(dtype, kv):
    inp = _batch(dtype, kv, 128, 16, 4, 2, [100, 3], [0, 0], 20, mask=None)
    inp["query"] = torch.zeros(5, 4, 128, dtype=DT[dtype])
    out = torch.full((5, 4, 128), 3.0, dtype=DT[dtype], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _run(inp, out=out, err=err)
    assert bool((out == 3).all()) and int(err) == 0


@pytest.mark.parametrize("kv", ["auto", "fp8_e4m3"])
def test_a_copy_that_never_arrives_is_reported(kv):
    """Every key stage of one launch expects 16 bytes more than arrive: its waits
    run into the (short) limit, the launch ends and says so, the next one is right."""
    inp = _batch("bf16", kv, 128, 16, 8, 2, [700, 40], [5, 3], 21)
    good = _run(inp)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_wait_limit_ns(20_000_000)
    try:
        pkv._test_set_unarrived_bytes(16)
        _run(inp, err=err)
        torch.cuda.synchronize()
    finally:
        pkv._test_set_unarrived_bytes(0)
        pkv.set_wait_limit_ns(0)
    assert int(err) & pkv.PKV_ERRF_TIMEOUT
    err.zero_()
    assert torch.equal(_run(inp, err=err), good) and int(err) == 0


def test_streams_graphs_and_shared_workspace():
    """Two captured graphs that share a workspace, replayed in turn; calls on two
    streams with a workspace each."""
    a = _batch("bf16", "auto", 128, 16, 8, 2, [3000], [5], 14)
    b = _batch("bf16", "fp8_e4m3", 128, 16, 8, 1, [2000, 77], [9, 4], 15)
    ws = _workspace(128)
    want = [_run(a).clone(), _run(b).clone()]
    gs, outs = [], []
    for inp in (a, b):
        g = on_device(inp)
        out = torch.zeros_like(g["query"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_attention_tree(out, g["query"], g["key_cache"], g["value_cache"], g["block_tables"],
                                     g["seq_lens"], g["cu"], g["scale"], workspace=ws, **_kwargs(g))
        gs.append((graph, g))
        outs.append(out)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for graph, _g in gs:
            graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [_workspace(128), _workspace(128)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (graph, g), o, s, w in zip(gs, outs, streams, spaces):
            with torch.cuda.stream(s):
                pkv.paged_attention_tree(o, g["query"], g["key_cache"], g["value_cache"], g["block_tables"],
                                         g["seq_lens"], g["cu"], g["scale"], workspace=w, **_kwargs(g))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("dtype,kv", [("bf16", "auto"), ("bf16", "fp8_e4m3"), ("f32", "auto")])
def test_a_verification_step_from_end_to_end(dtype, kv):
    """Write the drafted tokens into the cache, attend from the tree, accept a
    path, move its tokens together (read and write), decode the next token:
    as decoding the accepted tokens one after the other."""
    H, Hk, D, bs, ctx, T = 8, 2, 128, 16, 61, 7
    inp = _batch(dtype, kv, D, bs, H, Hk, [ctx + T + 1], [T], 16)
    parent = [-1, 0, 0, 1, 2, 4, 3]
    mask = torch.zeros(T, T, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            mask[i] = mask[p]
        mask[i, i] = True
    inp["mask"], inp["positions"] = mask, None
    path = [0, 2, 4, 5]
    g = on_device(inp)
    gen = torch.Generator().manual_seed(1)
    key, value = (torch.randn(T, Hk, D, generator=gen).to(DT[dtype]).cuda() for _ in range(2))
    table = g["block_tables"]

    def slots(first, n):
        pos = torch.arange(first, first + n, device="cuda")
        return table[0, pos // bs].long() * bs + pos % bs

    kw = dict(kv_cache_dtype=kv, k_scale=0.03, v_scale=0.04)
    ws = _workspace(D)
    kc, vc = g["key_cache"], g["value_cache"]
    pkv.paged_kv_write(kc, vc, key, value, slots(ctx, T), **kw)
    lens = torch.tensor([ctx + T], dtype=torch.int32, device="cuda")
    out = torch.empty_like(g["query"])
    pkv.paged_attention_tree(out, g["query"], kc, vc, table, lens, g["cu"], g["scale"], workspace=ws,
                             tree_mask=g["mask"], **kw)
    # move the accepted tokens behind the context
    ko, vo = torch.empty_like(key), torch.empty_like(value)
    pkv.paged_kv_read(ko, vo, kc, vc, table, torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                      seq_starts=torch.tensor([ctx], dtype=torch.int32, device="cuda"), **kw)
    pick = torch.tensor(path, device="cuda")
    pkv.paged_kv_write(kc, vc, ko[pick], vo[pick], slots(ctx, len(path)), **kw)
    for i, node in enumerate(path):
        step = torch.empty(1, H, D, dtype=DT[dtype], device="cuda")
        pkv.paged_attention_decode(step, g["query"][node:node + 1].contiguous(), kc, vc, table,
                                   torch.tensor([ctx + i + 1], dtype=torch.int32, device="cuda"), g["scale"], **kw)
        # both are within their bound of the exact result, which is the same
        ref = oracle.decode_v1(g["query"][node:node + 1].cpu(), kc.cpu(), vc.cpu(), inp["block_tables"],
                               [ctx + i + 1], inp["scale"], **kw)
        assert_attention_close(step, ref, DT[dtype], "decode")
        assert_attention_close(out[node:node + 1], ref, DT[dtype], f"node {node}")


def test_one_drafted_token_matches_decode():
    inp = _batch("bf16", "auto", 128, 16, 32, 8, [1, 500, 77, 2048], [1, 1, 1, 1], 17, mask=None)
    g = on_device(inp)
    dec = torch.empty_like(g["query"])
    pkv.paged_attention_decode(dec, g["query"], g["key_cache"], g["value_cache"], g["block_tables"],
                               g["seq_lens"], g["scale"])
    ref = _oracle(inp)
    assert_attention_close(_run(inp), ref, torch.bfloat16, "tree")
    assert_attention_close(dec, ref, torch.bfloat16, "decode")


def test_binding_refusals():
    inp = _batch("bf16", "auto", 128, 16, 8, 2, [100], [4], 18)
    with pytest.raises(ValueError, match="tree_mask"):
        _run(inp, tree_mask=torch.zeros(4, 4, device="cuda"))
    with pytest.raises(ValueError, match="tree_mask"):
        _run(inp, tree_mask=torch.zeros(3, 4, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError, match="positions"):
        _run(inp, positions=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="positions"):
        _run(inp, positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="cu_query_lens"):
        _run({**inp, "cu": torch.zeros(5, dtype=torch.int32)})
    with pytest.raises(ValueError, match="out must match"):
        _run(inp, out=torch.zeros(4, 8, 128, device="cuda"))
    with pytest.raises(RuntimeError, match="invalid"):
        _run(inp, workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError, match="invalid"):
        _run(inp, workspace=_workspace(128)[1:])
    with pytest.raises(RuntimeError, match="invalid"):
        _run(inp, cap=-1.0)
    with pytest.raises(ValueError, match="belong together"):
        g = on_device(inp)
        pkv.paged_attention_tree(g["query"], g["query"], g["key_cache"][:, :, :8], g["value_cache"],
                                 g["block_tables"], g["seq_lens"], g["cu"], 1.0, workspace=_workspace(128))
    empty = {**inp, "query": inp["query"][:0], "cu": torch.zeros(2, dtype=torch.int32), "mask": None,
             "positions": None}
    assert _run(empty).numel() == 0
