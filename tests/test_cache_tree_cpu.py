"""Cache write, cache read and tree attention without a GPU: the oracle is
pinned to independent statements of the definitions, and the library refuses
bad calls before it touches the CUDA runtime."""
import ctypes
import math

import pytest
import torch

import oracle
import workloads


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_tables_gb300 import _build
    try:
        _build.nvcc_path()
    except RuntimeError:
        pytest.skip("no CUDA toolkit")
    _build.build()
    import paged_kv_decode_tables_gb300 as pkv
    return pkv.lib()


# ------------------------------------------------------------------ oracle ---

@pytest.mark.parametrize("fmt,dt,top", [("e4m3", torch.float8_e4m3fn, 448.0),
                                        ("e5m2", torch.float8_e5m2, 57344.0)])
def test_encode_matches_torch_and_saturates(fmt, dt, top):
    g = torch.Generator().manual_seed(1)
    y = torch.randn(4000, generator=g) * torch.pow(2.0, torch.randint(-20, 18, (4000,), generator=g))
    codes = oracle.fp8.decode(torch.arange(128, dtype=torch.uint8), fmt)
    codes = codes[torch.isfinite(codes)]
    ties = ((codes[1:] + codes[:-1]) / 2).float()  # exact in float32
    y = torch.cat([y, ties, -ties, codes.float(), torch.tensor([0.0, -0.0, 1e30, -1e30, math.inf])])
    assert torch.equal(oracle.encode(y, fmt), y.clamp(-top, top).to(dt).view(torch.uint8))
    assert bool(torch.isnan(oracle.fp8.decode(oracle.encode(torch.tensor([math.nan]), fmt), fmt)))


@pytest.mark.parametrize("kv", ["auto", "fp8_e4m3"])
def test_what_is_written_is_read_back(kv):
    inp = workloads.make_inputs(num_heads=4, num_kv_heads=2, head_size=64, block_size=8, dtype="bf16",
                                seq_lens=[21, 5], seed=1, kv_cache_dtype=kv)
    n = 9
    g = torch.Generator().manual_seed(2)
    key = torch.randn(n, 2, 64, generator=g).bfloat16()
    value = torch.randn(n, 2, 64, generator=g).bfloat16()
    pos = torch.arange(12, 21)
    slots = inp["block_tables"][0, pos // 8].long() * 8 + pos % 8
    k2, v2 = oracle.kv_write(inp["key_cache"], inp["value_cache"], key, value, slots, kv, 0.05, 0.1)
    got = oracle.kv_read(torch.zeros(n, 2, 64).bfloat16(), torch.zeros(n, 2, 64).bfloat16(), k2, v2,
                         inp["block_tables"], [0, n, n], [12, 0], kv_cache_dtype=kv, k_scale=0.05,
                         v_scale=0.1)
    for x, y in zip(got, (key, value)):
        if kv == "auto":
            assert torch.equal(x, y)
        else:  # half a step of E4M3 (2^-4 of the value; its subnormal step is 2^-9) and one bf16 rounding
            assert bool(((x - y).abs().float() <= y.abs().float() * (2.0 ** -4 + 2.0 ** -8) + 0.1 * 2.0 ** -10).all())
    # and no other slot has changed
    keep = torch.ones(k2.shape[0] * 8, dtype=torch.bool)
    keep[slots] = False
    keep = keep.view(-1, 8)
    assert torch.equal(k2.permute(0, 3, 1, 2, 4)[keep], inp["key_cache"].permute(0, 3, 1, 2, 4)[keep])
    assert torch.equal(v2.permute(0, 3, 1, 2)[keep], inp["value_cache"].permute(0, 3, 1, 2)[keep])


def test_one_drafted_token_is_a_decode_step():
    inp = workloads.make_inputs(num_heads=4, num_kv_heads=2, head_size=64, block_size=8, dtype="f32",
                                seq_lens=[21, 5, 1], seed=3, alibi=True)
    args = (inp["query"], inp["key_cache"], inp["value_cache"], inp["block_tables"], inp["seq_lens_list"])
    slopes = inp["alibi_slopes"].tolist()
    ref = oracle.decode_v1(*args, inp["scale"], alibi_slopes=slopes)
    got = oracle.tree_attention(*args, [0, 1, 2, 3], inp["scale"], alibi_slopes=slopes)
    assert float((got - ref).abs().max()) < 1e-12


def test_chain_rows_are_decode_steps_of_shorter_sequences():
    inp = workloads.make_inputs(num_heads=4, num_kv_heads=2, head_size=64, block_size=8, dtype="f32",
                                seq_lens=[21], seed=4)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(6, 4, 64, generator=g)
    cache = (inp["key_cache"], inp["value_cache"], inp["block_tables"])
    got = oracle.tree_attention(q, *cache, [21], [0, 6], inp["scale"], logits_soft_cap=1e9)
    tri = oracle.tree_attention(q, *cache, [21], [0, 6], inp["scale"],
                                tree_mask=torch.tril(torch.ones(6, 6)).bool())
    for i in range(6):
        ref = oracle.decode_v1(q[i:i + 1], *cache, [16 + i], inp["scale"])
        assert float((got[i] - ref[0]).abs().max()) < 1e-9  # a cap of 1e9 changes nothing above 1e-12
        assert float((tri[i] - ref[0]).abs().max()) < 1e-12


# ----------------------------------------------------------------- refusals ---

def _cache_fields(a, dtype=2, x=8):
    a.num_kv_heads, a.head_size, a.block_size, a.x, a.num_blocks = 2, 128, 16, x, 32
    a.dtype, a.k_scale, a.v_scale = dtype, 1.0, 1.0
    a.key_cache = a.value_cache = 0x1000
    a.k_stride[:] = [2 * 16 * 128, 16 * 128, 16 * x, x, 1]
    a.v_stride[:] = [2 * 128 * 16, 128 * 16, 16, 1]
    a.key_stride[:] = a.value_stride[:] = [256, 128, 1]


def _write(lib, set_=None, **kw):
    import paged_kv_decode_tables_gb300 as pkv
    a = pkv.CacheWriteArgs()
    _cache_fields(a)
    a.num_tokens, a.key, a.value, a.slot_mapping, a.slot_stride = 3, 0x4000, 0x4000, 0x5000, 1
    for k, v in kw.items():
        setattr(a, k, v)
    if set_:
        set_(a)
    return lib.paged_kv_write(ctypes.byref(a), None)


def _read(lib, set_=None, **kw):
    import paged_kv_decode_tables_gb300 as pkv
    a = pkv.CacheReadArgs()
    _cache_fields(a)
    a.num_tokens, a.num_seqs, a.max_blocks_per_seq = 3, 1, 4
    a.key_out, a.value_out, a.block_tables, a.cu_seq_lens = 0x4000, 0x4000, 0x5000, 0x6000
    a.bt_stride[:] = [4, 1]
    for k, v in kw.items():
        setattr(a, k, v)
    if set_:
        set_(a)
    return lib.paged_kv_read(ctypes.byref(a), None)


SHARED_REFUSALS = [
    (dict(dtype=7), 1), (dict(kv_cache_dtype=3), 1), (dict(x=4), 1), (dict(num_tokens=-1), 1),
    (dict(num_kv_heads=0), 1), (dict(num_blocks=0), 1), (dict(head_size=96), 2),
    (dict(head_size=512), 2), (dict(block_size=24), 2), (dict(num_kv_heads=70000), 2),
    (dict(key_cache=None), 1), (dict(value_cache=0x1008), 1), (dict(key_cache=0x1008), 1),
    (dict(kv_cache_dtype=1, x=16, dtype=0), 2), (dict(kv_cache_dtype=1, x=16, k_scale=0.0), 1),
    (dict(kv_cache_dtype=1, x=16, v_scale=-1.0), 1),
    (dict(kv_cache_dtype=2, x=16, v_scale=float("nan")), 1),
]


@pytest.mark.parametrize("kw,status", SHARED_REFUSALS)
def test_cache_calls_refuse(lib, kw, status):
    assert _write(lib, **kw) == status
    assert _read(lib, **kw) == status


def test_cache_calls_refuse_layouts(lib):
    def stride(name, i, v):
        return lambda a: getattr(a, name).__setitem__(i, v)

    for call in (_write, _read):
        assert call(lib, stride("key_stride", 2, 2)) == 2   # elements of a head apart
        assert call(lib, stride("value_stride", 2, 0)) == 2
        assert call(lib, stride("k_stride", 3, 16)) == 2    # page not contiguous
        assert call(lib, stride("v_stride", 2, 32)) == 2
        assert call(lib, stride("v_stride", 0, 4100)) == 1  # block stride off 16 bytes
    assert lib.paged_kv_write(None, None) == 1 and lib.paged_kv_read(None, None) == 1
    assert _write(lib, key=None) == 1 and _write(lib, value=0x4001) == 1
    assert _write(lib, slot_mapping=None) == 1
    assert _read(lib, key_out=None) == 1 and _read(lib, block_tables=None) == 1
    assert _read(lib, cu_seq_lens=None) == 1 and _read(lib, num_seqs=-1) == 1
    assert _read(lib, num_seqs=65536) == 2 and _read(lib, max_blocks_per_seq=-1) == 1
    # nothing to do: no pointer is needed
    assert _write(lib, num_tokens=0, key=None, value=None, slot_mapping=None) == 0
    assert _read(lib, num_tokens=0, key_out=None, value_out=None) == 0
    assert _read(lib, num_seqs=0) == 0


def _tree(lib, decode=None, out=0x3000, **kw):
    import paged_kv_decode_tables_gb300 as pkv
    from test_abi import _args
    a = _args(**(decode or {}))
    t = pkv.TreeArgs()
    t.num_tokens, t.cu_query_lens, t.workspace = 5, 0x4000, 0x10000
    t.workspace_bytes = lib.pkv_tree_workspace_bytes(128)
    for k, v in kw.items():
        setattr(t, k, v)
    strides = (ctypes.c_int64 * 3)(8 * 128, 128, 1)
    return lib.paged_attention_tree(out, strides, ctypes.byref(a), ctypes.byref(t), None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), 1), (dict(mask_cols=-1), 1), (dict(cu_query_lens=None), 1),
    (dict(workspace=None), 1), (dict(workspace=0x10010), 1), (dict(workspace_bytes=1024), 1),
    (dict(logits_soft_cap=-1.0), 1), (dict(logits_soft_cap=float("inf")), 1),
    (dict(logits_soft_cap=float("nan")), 1), (dict(num_tokens=0x7fffffff), 2),
    (dict(decode=dict(head_size=96)), 2), (dict(decode=dict(scale=float("nan"))), 1),
    (dict(decode=dict(query=None)), 1), (dict(decode=dict(num_seqs=65536)), 2), (dict(out=None), 1),
])
def test_tree_refuses(lib, kw, status):
    assert _tree(lib, **kw) == status


def test_tree_with_nothing_to_do(lib):
    assert _tree(lib, num_tokens=0, decode=dict(query=None)) == 0
    assert _tree(lib, decode=dict(num_seqs=0)) == 0
    strides = (ctypes.c_int64 * 3)(8 * 128, 128, 1)
    assert lib.paged_attention_tree(0x3000, strides, None, None, None) == 1


def test_binding_refuses_cpu_tensors():
    import paged_kv_decode_tables_gb300 as pkv
    k = torch.zeros(4, 2, 8, 8, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_write(k, k, k, k, k)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_read(k, k, k, k, k, k)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_tree(k, k, k, k, k, k, k, 1.0, workspace=k)
