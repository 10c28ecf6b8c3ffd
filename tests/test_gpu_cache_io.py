"""Writing tokens into the paged caches and reading them back on the GPU,
against the slot-by-slot oracle.  Both are copies, quantisations to the
nearest code or one fp32 product rounded once, so every comparison is exact."""
import math

import pytest
import torch

import oracle
import paged_kv_decode_tables_gb300 as pkv
import workloads

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from paged_kv_decode_tables_gb300 import _build
    _build.build()


CASES = [
    # dtype, kv_cache_dtype, D, bs, Hk
    ("bf16", "auto", 128, 16, 8),
    ("f16", "auto", 64, 8, 3),
    ("f32", "auto", 128, 32, 2),
    ("f32", "auto", 64, 8, 1),
    ("bf16", "auto", 256, 32, 1),
    ("bf16", "fp8_e4m3", 128, 16, 4),
    ("f16", "fp8_e5m2", 64, 8, 5),
    ("bf16", "fp8_e5m2", 256, 32, 2),
    ("f16", "fp8", 128, 8, 1),
]


def _batch(dtype, kv, D, bs, Hk, lens, seed, **kw):
    return workloads.make_inputs(num_heads=Hk, num_kv_heads=Hk, head_size=D, block_size=bs,
                                 dtype=dtype, seq_lens=lens, seed=seed, kv_cache_dtype=kv,
                                 k_scale=0.037, v_scale=0.21, **kw)


def _tokens(n, Hk, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, Hk, D, generator=g).to(DT[dtype]),
            torch.randn(n, Hk, D, generator=g).to(DT[dtype]))


def _slots(inp, spans):
    """Slots of tokens [a, b) of sequence s, one span behind the other."""
    bs, out = inp["block_size"], []
    for s, a, b in spans:
        pos = torch.arange(a, b)
        out.append(inp["block_tables"][s, pos // bs].long() * bs + pos % bs)
    return torch.cat(out)


def _same(a, b):
    """Equal values and the same bits of every number (NaN equals NaN)."""
    if a.dtype == torch.uint8:
        return torch.equal(a, b)
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def _check_write(inp, key, value, slots, kv):
    kc, vc = inp["key_cache"].cuda(), inp["value_cache"].cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_kv_write(kc, vc, key.cuda(), value.cuda(), slots.cuda(), kv_cache_dtype=kv,
                       k_scale=inp["k_scale"], v_scale=inp["v_scale"], err_flag=err)
    rk, rv = oracle.kv_write(inp["key_cache"], inp["value_cache"], key, value, slots, kv,
                             inp["k_scale"], inp["v_scale"])
    assert _same(kc.cpu(), rk) and _same(vc.cpu(), rv)
    assert int(err) == 0


@pytest.mark.parametrize("dtype,kv,D,bs,Hk", CASES)
def test_write_prompts_and_steps(dtype, kv, D, bs, Hk):
    lens = [70, 1, 33, 8, 45]
    inp = _batch(dtype, kv, D, bs, Hk, lens, D + bs + Hk)
    # whole prompts, a middle piece off the 8-token grid, single tokens, padding between and behind
    spans = [(0, 0, 70), (1, 0, 1), (2, 5, 30), (3, 7, 8), (4, 44, 45), (4, 3, 4)]
    slots = _slots(inp, spans)
    slots = torch.cat([slots[:9], torch.tensor([-1]), slots[9:], torch.tensor([-1, -5])])
    key, value = _tokens(len(slots), Hk, D, dtype, 3)
    _check_write(inp, key, value, slots, kv)


@pytest.mark.parametrize("kv", ["auto", "fp8_e4m3"])
def test_write_any_order(kv):
    """Slots in random order, so no run of eight stands together."""
    inp = _batch("bf16", kv, 64, 8, 2, [61], 1)
    slots = _slots(inp, [(0, 0, 61)])[torch.randperm(61, generator=torch.Generator().manual_seed(4))]
    key, value = _tokens(61, 2, 64, "bf16", 5)
    _check_write(inp, key, value, slots, kv)


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 257])
def test_write_lengths(n):
    inp = _batch("bf16", "fp8_e4m3", 128, 16, 2, [300], 2)
    key, value = _tokens(n, 2, 128, "bf16", n)
    _check_write(inp, key, value, _slots(inp, [(0, 11, 11 + n)]), "fp8_e4m3")


@pytest.mark.parametrize("kv", ["fp8_e4m3", "fp8_e5m2"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_write_special_values(kv, dtype):
    """Infinities saturate, NaN stays NaN, ties go to the even code, subnormals and zeros of both signs."""
    inp = _batch(dtype, kv, 64, 16, 1, [16], 3)
    inp["k_scale"], inp["v_scale"] = 1.0, 0.5
    codes = oracle.fp8.decode(torch.arange(256, dtype=torch.uint8), oracle.fp8.format_of(kv))
    codes = codes[torch.isfinite(codes)].sort().values
    special = torch.cat([codes, (codes[1:] + codes[:-1]) / 2,
                         torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 449.0, 6e4, -6e4]).double()])
    special = special.to(DT[dtype])
    key = torch.zeros(16, 1, 64, dtype=DT[dtype])
    key.flatten()[:special.numel()] = special
    kc, vc = inp["key_cache"].cuda(), inp["value_cache"].cuda()
    slots = _slots(inp, [(0, 0, 16)])
    pkv.paged_kv_write(kc, vc, key.cuda(), key.cuda(), slots.cuda(), kv_cache_dtype=kv, k_scale=1.0,
                       v_scale=0.5)
    rk, rv = oracle.kv_write(inp["key_cache"], inp["value_cache"], key, key, slots, kv, 1.0, 0.5)
    fmt = oracle.fp8.format_of(kv)
    for a, b in ((kc.cpu(), rk), (vc.cpu(), rv)):
        x, y = oracle.fp8.decode(a, fmt), oracle.fp8.decode(b, fmt)
        assert torch.equal(torch.isnan(x), torch.isnan(y))
        ok = ~torch.isnan(x)
        assert torch.equal(a[ok], b[ok])


@pytest.mark.parametrize("kv", ["fp8_e4m3", "fp8_e5m2"])
@pytest.mark.parametrize("scale", [1.0, 0.25, 0.1, 3.0, 0.043, 0.0271, 7.3e-18, 1.1e18, 1.0 / 3.0, 7e-39, 2.0 ** -130, 3e38, 1.1754944e-38])
def test_every_half_precision_value_and_scale(kv, scale):
    """All fp16 numbers over scales that are powers of two, round to them, have
    no normal reciprocal: the code is that of the fp32 quotient, ties included."""
    n = 1024
    key = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16).view(n, 1, 64).contiguous()
    inp = _batch("f16", kv, 64, 16, 1, [n], 4)
    kc, vc = inp["key_cache"].cuda(), inp["value_cache"].cuda()
    slots = _slots(inp, [(0, 0, n)])
    pkv.paged_kv_write(kc, vc, key.cuda(), key.cuda(), slots.cuda(), kv_cache_dtype=kv, k_scale=scale, v_scale=scale)
    want = oracle.encode(key.float() / torch.tensor(scale, dtype=torch.float32), oracle.fp8.format_of(kv))
    rows = kc.cpu().permute(0, 3, 1, 2, 4).reshape(-1, 1, 64)[slots], vc.cpu().permute(0, 3, 1, 2).reshape(-1, 1, 64)[slots]
    nan = torch.isnan(key)
    for got in rows:
        assert torch.equal(got[~nan], want[~nan])
        assert bool(torch.isnan(oracle.fp8.decode(got[nan], oracle.fp8.format_of(kv))).all())


@pytest.mark.parametrize("dtype,kv,D,bs,Hk", CASES)
@pytest.mark.parametrize("start", [0, 1, 13])
def test_read(dtype, kv, D, bs, Hk, start):
    lens = [40, 0, 1, 16, 70, 0]
    inp = _batch(dtype, kv, D, bs, Hk, [n + start for n in lens], D + Hk, bt_col_step=2,
                 unused_slot_fill=math.nan)
    cu = torch.tensor([0] + lens).cumsum(0).int()
    n = int(cu[-1]) + 3  # rows behind the last sequence stay as they were
    starts = torch.tensor([start] * len(lens), dtype=torch.int32)
    ko, vo = _tokens(n, Hk, D, dtype, 9)
    kg, vg = ko.cuda(), vo.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = inp["block_tables_storage"].cuda()[:, ::2]
    pkv.paged_kv_read(kg, vg, inp["key_cache"].cuda(), inp["value_cache"].cuda(), table,
                      cu.cuda(), seq_starts=starts.cuda() if start else None, kv_cache_dtype=kv,
                      k_scale=inp["k_scale"], v_scale=inp["v_scale"], err_flag=err)
    rk, rv = oracle.kv_read(ko, vo, inp["key_cache"], inp["value_cache"], inp["block_tables"], cu,
                            starts, kv_cache_dtype=kv, k_scale=inp["k_scale"], v_scale=inp["v_scale"])
    assert torch.equal(kg.cpu(), rk) and torch.equal(vg.cpu(), rv)
    assert int(err) == 0
    # the flat page list of the page-index copy instead of the table
    nblk = [len(r) for r in inp["block_rows"]]
    indptr = torch.tensor([0] + nblk).cumsum(0).int().cuda()
    pages = torch.tensor(sum(inp["block_rows"], []), dtype=torch.int32).cuda()
    kg2, vg2 = ko.cuda(), vo.cuda()
    pkv.paged_kv_read(kg2, vg2, inp["key_cache"].cuda(), inp["value_cache"].cuda(), pages, cu.cuda(),
                      seq_starts=starts.cuda(), kv_indptr=indptr, kv_cache_dtype=kv,
                      k_scale=inp["k_scale"], v_scale=inp["v_scale"], err_flag=err)
    assert torch.equal(kg2, kg) and torch.equal(vg2, vg) and int(err) == 0


@pytest.mark.parametrize("B", [1, 2, 33, 300])
def test_read_many_sequences(B):
    """The search over cu_seq_lens: empty and one-token sequences among longer ones."""
    lens = [(7 * i * i) % 23 if i % 3 else i % 2 for i in range(B)]
    inp = _batch("bf16", "auto", 64, 8, 2, lens, B)
    cu = torch.tensor([0] + lens).cumsum(0).int()
    n = max(1, int(cu[-1]))
    ko, vo = _tokens(n, 2, 64, "bf16", 1)
    kg, vg = ko.cuda(), vo.cuda()
    pkv.paged_kv_read(kg, vg, inp["key_cache"].cuda(), inp["value_cache"].cuda(),
                      inp["block_tables"].cuda(), cu.cuda())
    rk, rv = oracle.kv_read(ko, vo, inp["key_cache"], inp["value_cache"], inp["block_tables"], cu)
    assert torch.equal(kg.cpu(), rk) and torch.equal(vg.cpu(), rv)


@pytest.mark.parametrize("kv", ["auto", "fp8_e4m3"])
def test_strided_and_unaligned_views(kv):
    """Keys and values as views of a joint projection (aligned), and of one whose
    rows are off the 16-byte grid; caches with gaps between blocks and heads."""
    inp = _batch("bf16", kv, 64, 16, 3, [50], 6)
    slots = _slots(inp, [(0, 0, 50)])
    nb, _, c, bs, x = inp["key_cache"].shape
    wide_k = torch.zeros(nb, 5, c + 1, bs, x, dtype=inp["key_cache"].dtype)
    wide_v = torch.zeros(nb, 4, 64 + 8, bs, dtype=inp["value_cache"].dtype)
    wide_k[:, :3, :c], wide_v[:, 1:, :64] = inp["key_cache"], inp["value_cache"]
    for pad in (0, 1):
        joint = torch.randn(50, 7, 64 + pad, generator=torch.Generator().manual_seed(8)).bfloat16()
        key, value = joint[:, 1:4, pad:], joint[:, 4:, pad:]
        wk, wv = wide_k.clone().cuda(), wide_v.clone().cuda()
        j = joint.cuda()
        pkv.paged_kv_write(wk[:, :3, :c], wv[:, 1:, :64], j[:, 1:4, pad:], j[:, 4:, pad:], slots.cuda(),
                           kv_cache_dtype=kv, k_scale=inp["k_scale"], v_scale=inp["v_scale"])
        rk, rv = oracle.kv_write(inp["key_cache"], inp["value_cache"], key, value, slots, kv,
                                 inp["k_scale"], inp["v_scale"])
        assert torch.equal(wk[:, :3, :c].cpu(), rk) and torch.equal(wv[:, 1:, :64].cpu(), rv)
        assert bool((wk[:, 3:] == 0).all()) and bool((wk[:, :3, c:] == 0).all())
        assert bool((wv[:, :1] == 0).all()) and bool((wv[:, 1:, 64:] == 0).all())
        back = torch.zeros_like(j)
        cu = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
        pkv.paged_kv_read(back[:, 1:4, pad:], back[:, 4:, pad:], wk[:, :3, :c], wv[:, 1:, :64],
                          inp["block_tables"].cuda(), cu, kv_cache_dtype=kv, k_scale=inp["k_scale"],
                          v_scale=inp["v_scale"])
        ek, ev = oracle.kv_read(torch.zeros(50, 3, 64).bfloat16(), torch.zeros(50, 3, 64).bfloat16(),
                                rk, rv, inp["block_tables"], [0, 50], kv_cache_dtype=kv,
                                k_scale=inp["k_scale"], v_scale=inp["v_scale"])
        assert torch.equal(back[:, 1:4, pad:].cpu(), ek) and torch.equal(back[:, 4:, pad:].cpu(), ev)
        assert bool((back[:, 0] == 0).all()) and (pad == 0 or bool((back[..., 0] == 0).all()))


def test_bad_device_data_is_flagged_and_skipped():
    inp = _batch("bf16", "auto", 64, 8, 2, [20, 20], 7)
    kc, vc = inp["key_cache"].cuda(), inp["value_cache"].cuda()
    key, value = _tokens(3, 2, 64, "bf16", 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, kc.shape[0] * 8, 2 ** 40])
    pkv.paged_kv_write(kc, vc, key.cuda(), value.cuda(), slots.cuda(), err_flag=err)
    assert int(err) == pkv.PKV_ERRF_BLOCK_ID
    rk, rv = oracle.kv_write(inp["key_cache"], inp["value_cache"], key, value, slots)
    assert torch.equal(kc.cpu(), rk) and torch.equal(vc.cpu(), rv)

    def read(cu, starts=None, table=None, n=20):
        ko = torch.full((n, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        vo = ko.clone()
        e = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.paged_kv_read(ko, vo, kc, vc, (inp["block_tables"] if table is None else table).cuda(),
                          torch.tensor(cu, dtype=torch.int32, device="cuda"), err_flag=e,
                          seq_starts=None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda())
        return ko, int(e)

    ko, e = read([0, 20, 25])      # the second sequence leaves the output
    assert e == pkv.PKV_ERRF_INDPTR
    ko, e = read([0, 20], [10])    # tokens 10..29 of a row of three pages of 8
    assert e == pkv.PKV_ERRF_SEQ_LEN and bool((ko[14:] == 5).all()) and not bool((ko[:14] == 5).any())
    ko, e = read([0, 20], [-3])
    assert e == pkv.PKV_ERRF_SEQ_LEN and bool((ko == 5).all())
    bad = inp["block_tables"].clone()
    bad[0, 1] = kc.shape[0]
    ko, e = read([0, 20], None, bad)
    assert e == pkv.PKV_ERRF_BLOCK_ID


def test_streams_and_graph_replay():
    """A call on a stream of its own, and write + read captured into a graph and replayed on new tokens."""
    inp = _batch("bf16", "fp8_e4m3", 128, 16, 2, [90], 8)
    kc, vc, table = inp["key_cache"].cuda(), inp["value_cache"].cuda(), inp["block_tables"].cuda()
    key, value = (t.cuda() for t in _tokens(30, 2, 128, "bf16", 1))
    slots = _slots(inp, [(0, 60, 90)]).cuda()
    cu = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
    starts = torch.tensor([60], dtype=torch.int32, device="cuda")
    ko, vo = torch.zeros_like(key), torch.zeros_like(value)
    kw = dict(kv_cache_dtype="fp8_e4m3", k_scale=0.05, v_scale=0.05)

    def both():
        pkv.paged_kv_write(kc, vc, key, value, slots, **kw)
        pkv.paged_kv_read(ko, vo, kc, vc, table, cu, seq_starts=starts, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    first = ko.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (2, 3):
        k2, v2 = _tokens(30, 2, 128, "bf16", seed)
        key.copy_(k2)
        value.copy_(v2)
        graph.replay()
        torch.cuda.synchronize()
        ek, ev = oracle.kv_write(inp["key_cache"], inp["value_cache"], k2, v2, slots.cpu(), "fp8_e4m3", 0.05, 0.05)
        rk, rv = oracle.kv_read(k2, v2, ek, ev, inp["block_tables"], [0, 30], [60], kv_cache_dtype="fp8_e4m3",
                                k_scale=0.05, v_scale=0.05)
        assert torch.equal(ko.cpu(), rk) and torch.equal(vo.cpu(), rv)
        assert not torch.equal(ko, first)


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: slots in its last block."""
    nb, hk, d, bs = 70000, 8, 256, 16
    kc = torch.zeros(nb, hk, d // 16, bs, 16, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(nb, hk, d, bs, dtype=torch.uint8, device="cuda")
    assert kc.numel() > 2 ** 31
    key, value = _tokens(16, hk, d, "bf16", 4)
    slots = torch.arange((nb - 1) * bs, nb * bs)
    kw = dict(kv_cache_dtype="fp8_e4m3", k_scale=0.25, v_scale=0.25)
    pkv.paged_kv_write(kc, vc, key.cuda(), value.cuda(), slots.cuda(), **kw)
    ko, vo = torch.zeros(16, hk, d).bfloat16().cuda(), torch.zeros(16, hk, d).bfloat16().cuda()
    pkv.paged_kv_read(ko, vo, kc, vc, torch.tensor([[nb - 1]], dtype=torch.int32).cuda(),
                      torch.tensor([0, 16], dtype=torch.int32).cuda(), **kw)
    rk, rv = oracle.kv_write(torch.zeros(1, hk, d // 16, bs, 16).byte(), torch.zeros(1, hk, d, bs).byte(),
                             key, value, torch.arange(16), "fp8_e4m3", 0.25, 0.25)
    assert torch.equal(kc[-1:].cpu(), rk) and torch.equal(vc[-1:].cpu(), rv)
    ek, ev = oracle.kv_read(key, value, rk, rv, torch.tensor([[0]]), [0, 16], kv_cache_dtype="fp8_e4m3",
                            k_scale=0.25, v_scale=0.25)
    assert torch.equal(ko.cpu(), ek) and torch.equal(vo.cpu(), ev)
    del kc, vc
    torch.cuda.empty_cache()


def test_binding_refusals():
    inp = _batch("bf16", "auto", 64, 8, 2, [20], 9)
    kc, vc = inp["key_cache"].cuda(), inp["value_cache"].cuda()
    key, value = (t.cuda() for t in _tokens(4, 2, 64, "bf16", 1))
    slots = torch.arange(4).cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32).cuda()
    table = inp["block_tables"].cuda()
    with pytest.raises(ValueError, match="slot_mapping"):
        pkv.paged_kv_write(kc, vc, key, value, slots.int())
    with pytest.raises(ValueError, match="slot_mapping"):
        pkv.paged_kv_write(kc, vc, key, value, slots[:3])
    with pytest.raises(ValueError, match="dtype"):
        pkv.paged_kv_write(kc, vc, key.half(), value, slots)
    with pytest.raises(ValueError, match="share a dtype"):
        pkv.paged_kv_write(kc, vc, key.half(), value.half(), slots)
    with pytest.raises(ValueError, match="for these caches"):
        pkv.paged_kv_write(kc, vc, key[:, :1], value[:, :1], slots)
    with pytest.raises(ValueError, match="belong together"):
        pkv.paged_kv_write(kc, vc[:, :1], key, value, slots)
    with pytest.raises(RuntimeError, match="unsupported"):
        pkv.paged_kv_write(kc, vc, key.transpose(1, 2).contiguous().transpose(1, 2), value, slots)
    with pytest.raises(ValueError, match="fp8 caches"):
        pkv.paged_kv_write(kc, vc, key, value, slots, kv_cache_dtype="fp8")
    with pytest.raises(ValueError, match="cu_seq_lens"):
        pkv.paged_kv_read(key, value, kc, vc, table, cu.long())
    with pytest.raises(ValueError, match="seq_starts"):
        pkv.paged_kv_read(key, value, kc, vc, table, cu, seq_starts=cu)
    with pytest.raises(ValueError, match="block_tables"):
        pkv.paged_kv_read(key, value, kc, vc, table[:0], cu)
    with pytest.raises(ValueError, match="columns"):
        pkv.paged_kv_read(key, value, kc, vc, table, cu, max_blocks_per_seq=99)
