"""Cases and plain forms of the paged-cache operators: writing tokens into the
cache (with 8-bit quantisation), reading sequences back out of it, and the
attention of drafted token trees over it.

``listed`` and ``draw`` name cases by plain numbers, ``prepare`` makes what a
serving program holds before the call, ``run`` is one call: the library's
kernels where ``own`` is true, elementary torch operations in 32 bits where it
is not.  ``exact`` restates the definition in 64 bits, sequence by sequence.

Cache layouts: ``key_cache [num_blocks, num_kv_heads, head_size / x,
block_size, x]`` with x = 16 bytes of elements, ``value_cache [num_blocks,
num_kv_heads, head_size, block_size]``.  The 8-bit caches hold codes; a code
stands for its format's value times the cache's scale.
"""
import math
import random

import torch

own = False

_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_FP8 = {"fp8_e4m3": torch.float8_e4m3fn, "fp8_e5m2": torch.float8_e5m2}
_FP8_MAX = {"fp8_e4m3": 448.0, "fp8_e5m2": 57344.0}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def _lib():
    import paged_kv_decode_tables_gb300
    return paged_kv_decode_tables_gb300


def listed():
    return [
        # The smallest step: four sequences append their token to a bf16 cache.
        dict(name="write_step_4_bf16", op="write", shape="step", seqs=4, least=40, most=900, dtype="bf16",
             kv="auto", kv_heads=8, head_size=128, block_size=16, pad=0),
        # A padded step of the ragged serving batch (512 sequences) into an E4M3 cache: the last rows
        # are padding with slot -1.
        dict(name="write_step_512_e4m3", op="write", shape="step", seqs=512, least=1, most=2048, dtype="bf16",
             kv="fp8_e4m3", kv_heads=8, head_size=128, block_size=16, pad=19),
        # Prompts of a prefill, packed one behind the other, into a bf16 cache.
        dict(name="write_prompts_bf16", op="write", shape="prompt", seqs=13, least=700, most=4500, dtype="bf16",
             kv="auto", kv_heads=8, head_size=128, block_size=16, pad=0),
        # fp16 prompts of a model with as many kv heads as heads, quantised to E5M2, 32-token pages.
        dict(name="write_prompts_f16_e5m2", op="write", shape="prompt", seqs=7, least=33, most=3001, dtype="f16",
             kv="fp8_e5m2", kv_heads=32, head_size=64, block_size=32, pad=5),
        # A cached prefix of two sequences read back for the rest of their prompt.
        dict(name="read_prefix_2_bf16", op="read", seqs=2, least=37, most=301, start=0, dtype="bf16", kv="auto",
             kv_heads=8, head_size=128, block_size=16),
        # Long contexts of an E4M3 cache read back as bf16, from the middle of a page on.
        dict(name="read_long_e4m3", op="read", seqs=9, least=2000, most=16385, start=45, dtype="bf16",
             kv="fp8_e4m3", kv_heads=8, head_size=128, block_size=16),
        # The smallest verification: one sequence, a tree of eight drafted tokens.
        dict(name="tree_1x8_bf16", op="tree", seqs=1, least=517, most=517, draft=8, fewest=8, dtype="bf16",
             kv="auto", heads=32, kv_heads=8, head_size=128, block_size=16, cap=0.0, alibi=False),
        # A ragged serving batch, each sequence with its own tree of up to 16 tokens.
        dict(name="tree_128x16_bf16", op="tree", seqs=128, least=64, most=8192, draft=16, fewest=1, dtype="bf16",
             kv="auto", heads=32, kv_heads=8, head_size=128, block_size=16, cap=0.0, alibi=False),
        # Long contexts, 64 query heads over 8 kv heads: 16 drafted tokens make 128 rows a kv head.
        dict(name="tree_8x16_long_bf16", op="tree", seqs=8, least=16384, most=131072, draft=16, fewest=16,
             dtype="bf16", kv="auto", heads=64, kv_heads=8, head_size=128, block_size=16, cap=0.0, alibi=False),
        # Wide trees (64 tokens, 256 rows a kv head) of a fp16 model whose scores are capped by a tanh.
        dict(name="tree_32x64_cap_f16", op="tree", seqs=32, least=200, most=4096, draft=64, fewest=40, dtype="f16",
             kv="auto", heads=16, kv_heads=4, head_size=256, block_size=16, cap=50.0, alibi=False),
        # An E4M3 cache under a model with a distance bias (ALiBi slopes, positions by tree depth).
        dict(name="tree_64x24_alibi_e4m3", op="tree", seqs=64, least=500, most=6000, draft=24, fewest=3, dtype="bf16",
             kv="fp8_e4m3", heads=32, kv_heads=8, head_size=128, block_size=16, cap=0.0, alibi=True),
        # fp32 all the way, a small model's batch, 8-token pages.
        dict(name="tree_16x5_f32", op="tree", seqs=16, least=13, most=2048, draft=5, fewest=2, dtype="f32", kv="auto",
             heads=8, kv_heads=4, head_size=64, block_size=8, cap=0.0, alibi=False),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["write", "read", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"] if op != "tree" else ["bf16", "bf16", "bf16", "f16", "f16", "f32"])
    kv = rng.choice(["auto", "auto", "fp8_e4m3", "fp8_e5m2"]) if dtype != "f32" else "auto"
    c = dict(op=op, dtype=dtype, kv=kv, block_size=rng.choice([8, 16, 16, 32]),
             head_size=rng.choice([64, 128, 128, 256] if dtype != "f32" else [64, 128]))
    if op == "write":
        if rng.random() < 0.5:
            c.update(shape="step", seqs=_log(rng, 1, 700), least=1, most=_log(rng, 10, 2000), pad=rng.randint(0, 9))
        else:
            c.update(shape="prompt", seqs=rng.randint(1, 9), least=_log(rng, 1, 50), pad=rng.randint(0, 3))
            c.update(most=c["least"] + _log(rng, 60, 2500))
        c.update(kv_heads=rng.randint(1, 12))
    elif op == "read":
        c.update(seqs=_log(rng, 1, 40), least=_log(rng, 1, 50), start=rng.choice([0, 0, 1, 33, 100]),
                 kv_heads=rng.randint(1, 10))
        c.update(most=c["least"] + _log(rng, 60, 3000))
    else:
        group = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
        c.update(seqs=_log(rng, 1, 40), kv_heads=rng.randint(1, 8 if group < 8 else 4), draft=_log(rng, 1, 64),
                 least=64, cap=rng.choice([0.0, 0.0, 0.0, 30.0]), alibi=rng.random() < 0.25)
        c.update(heads=group * c["kv_heads"], fewest=rng.randint(1, c["draft"]))
        longest = min(20000, 200000 // c["seqs"], int(2e11 / (4 * c["draft"] * c["heads"] * c["head_size"] * c["seqs"])))
        c.update(most=c["least"] + _log(rng, 20, longest))
    return c


def _lengths(case):
    """Token counts of the case's sequences: between `least` and `most`, both of them among the lengths
    where there is more than one sequence, spread over the logarithm."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["least"], case["most"]))
    got = [min(case["most"], max(case["least"], _log(rng, case["least"], case["most"]))) for _ in range(case["seqs"])]
    got[0] = case["most"]
    got[-1] = case["least"] if case["seqs"] > 1 else got[-1]
    return got


def _drafts(case):
    """Drafted tokens of each sequence, at most its whole length."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["draft"], case["fewest"]))
    return [min(n, rng.randint(case["fewest"], case["draft"])) for n in _lengths(case)]


def _x(case):
    return 16 if case["kv"] != "auto" else 16 // _SIZE[case["dtype"]]


def _cache_bytes(case):
    return 1 if case["kv"] != "auto" else _SIZE[case["dtype"]]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dtype, kv = _TORCH[case["dtype"]], case["kv"]
    hk, d, bs, x = case["kv_heads"], case["head_size"], case["block_size"], _x(case)
    lens = _lengths(case)
    starts = [case.get("start", 0)] * len(lens)
    pages = [-(-(n + s) // bs) for n, s in zip(lens, starts)]
    blocks = sum(pages) + max(2, sum(pages) // 16)  # a pool with a few blocks to spare
    k_scale, v_scale = (0.043, 0.027) if kv != "auto" else (1.0, 1.0)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def cache(*shape):
        if kv == "auto":
            return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float16) * 30).to(_FP8[kv]).view(torch.uint8)

    state = dict(case=case, key_cache=cache(blocks, hk, d // x, bs, x), value_cache=cache(blocks, hk, d, bs),
                 k_scale=k_scale, v_scale=v_scale)
    owned = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device=dev)  # -1: owned by no sequence
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = owned[at:at + n]
        at += n
    state["block_tables"] = table
    if case["op"] == "write":
        step = case["shape"] == "step"
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor([1 if step else n for n in lens])).to(dev)
        pos = torch.tensor([n - 1 for n in lens]) if step else torch.cat([torch.arange(n) for n in lens])
        pos = pos.to(dev)
        slots = table[seq, pos // bs].to(torch.int64) * bs + pos % bs
        slots = torch.cat([slots, torch.full((case["pad"],), -1, dtype=torch.int64, device=dev)])
        # keys and values are views of one projection's output, as a model's layer has them
        both = normal(slots.numel(), 2, hk, d)
        state.update(slots=slots, key=both[:, 0], value=both[:, 1])
    elif case["op"] == "read":
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
        total = sum(lens)
        state.update(cu_seq_lens=cu, seq_starts=torch.tensor(starts, dtype=torch.int32, device=dev),
                     key_out=torch.zeros(total, hk, d, dtype=dtype, device=dev),
                     value_out=torch.zeros(total, hk, d, dtype=dtype, device=dev))
    else:
        drafts, widest = _drafts(case), case["draft"]
        b = len(lens)
        count = torch.tensor(drafts, device=dev)
        # random trees: a node hangs below one of the eight before it, or starts a branch of its own
        parent = torch.arange(widest, device=dev) - 1 - torch.randint(0, 8, (b, widest), generator=gen, device=dev)
        mask = torch.zeros(b, widest, widest, dtype=torch.bool, device=dev)
        rows = torch.arange(b, device=dev)
        for i in range(widest):
            p = parent[:, i]
            mask[:, i] = mask[rows, p.clamp(min=0)] & (p >= 0)[:, None]
            mask[:, i, i] = True
        real = torch.arange(widest, device=dev)[None] < count[:, None]
        total = sum(drafts)
        ctx = torch.tensor([n - t for n, t in zip(lens, drafts)], device=dev)
        state.update(query=normal(total, case["heads"], d), out=torch.zeros(total, case["heads"], d, dtype=dtype, device=dev),
                     seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                     cu_query_lens=torch.tensor([0] + drafts).cumsum(0).to(torch.int32).to(dev),
                     tree_mask=mask[real].contiguous(), scale=d ** -0.5, positions=None, slopes=None)
        if case["alibi"]:
            state["positions"] = (ctx[:, None] + mask.sum(-1) - 1)[real].to(torch.int32)
            h = case["heads"]
            state["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device=dev)
    return state


# ------------------------------------------------------------ the library's calls --


def _own_write(s):
    kv = s["case"]["kv"]
    _lib().paged_kv_write(s["key_cache"], s["value_cache"], s["key"], s["value"], s["slots"], kv_cache_dtype=kv,
                          k_scale=s["k_scale"], v_scale=s["v_scale"])
    if kv == "auto":
        return dict(key_cache=s["key_cache"], value_cache=s["value_cache"])
    return dict(key_cache=s["key_cache"].view(_FP8[kv]), value_cache=s["value_cache"].view(_FP8[kv]))


def _own_read(s):
    _lib().paged_kv_read(s["key_out"], s["value_out"], s["key_cache"], s["value_cache"], s["block_tables"],
                         s["cu_seq_lens"], seq_starts=s["seq_starts"], kv_cache_dtype=s["case"]["kv"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
    return dict(key=s["key_out"], value=s["value_out"])


def _own_tree(s):
    lib, c = _lib(), s["case"]
    if "workspace" not in s:  # a serving program keeps one for all its calls
        s["workspace"] = torch.empty(lib.tree_workspace_bytes(c["head_size"]), dtype=torch.uint8, device="cuda")
    lib.paged_attention_tree(s["out"], s["query"], s["key_cache"], s["value_cache"], s["block_tables"],
                             s["seq_lens"], s["cu_query_lens"], s["scale"], workspace=s["workspace"],
                             tree_mask=s["tree_mask"], positions=s["positions"], logits_soft_cap=c["cap"],
                             kv_cache_dtype=c["kv"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                             alibi_slopes=s["slopes"])
    return s["out"]


# ------------------------------------------------------------------ the plain forms --


def _plain_write(s):
    case, kv = s["case"], s["case"]["kv"]
    bs, x = case["block_size"], _x(case)
    real = s["slots"] >= 0
    slots, key, value = s["slots"][real], s["key"][real], s["value"][real]
    if kv != "auto":
        top = _FP8_MAX[kv]
        key = (key.float() / s["k_scale"]).clamp(-top, top).to(_FP8[kv]).view(torch.uint8)
        value = (value.float() / s["v_scale"]).clamp(-top, top).to(_FP8[kv]).view(torch.uint8)
    n, hk, d = key.shape
    s["key_cache"][slots // bs, :, :, slots % bs, :] = key.reshape(n, hk, d // x, x)
    s["value_cache"][slots // bs, :, :, slots % bs] = value
    if kv == "auto":
        return dict(key_cache=s["key_cache"], value_cache=s["value_cache"])
    return dict(key_cache=s["key_cache"].view(_FP8[kv]), value_cache=s["value_cache"].view(_FP8[kv]))


def _plain_read(s):
    case, kv = s["case"], s["case"]["kv"]
    bs, dtype = case["block_size"], _TORCH[case["dtype"]]
    cu = s["cu_seq_lens"].long()
    row = torch.arange(s["key_out"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = row - cu[seq] + s["seq_starts"].long()[seq]
    block = s["block_tables"][seq, pos // bs].long()
    key, value = s["key_cache"][block, :, :, pos % bs, :].flatten(2), s["value_cache"][block, :, :, pos % bs]
    if kv != "auto":
        key = (key.view(_FP8[kv]).float() * s["k_scale"]).to(dtype)
        value = (value.view(_FP8[kv]).float() * s["v_scale"]).to(dtype)
    return dict(key=key, value=value)


def _plain_tree(s):
    case, kv = s["case"], s["case"]["kv"]
    hk, d, bs = case["kv_heads"], case["head_size"], case["block_size"]
    group = case["heads"] // hk
    cu, lens = s["cu_query_lens"].long(), s["seq_lens"].long()
    dev, b, widest = cu.device, lens.numel(), s["tree_mask"].shape[1]
    count = cu[1:] - cu[:-1]
    ctx = lens - count
    # queries and mask rows, padded to [sequences, widest]
    node = torch.arange(widest, device=dev)
    row = (cu[:-1, None] + node).clamp(max=s["query"].shape[0] - 1)
    q = s["query"].float()[row].view(b, widest, hk, group, d).permute(0, 2, 1, 3, 4).reshape(b, hk, widest * group, d)
    # keys and values through the block tables, [sequences, kv heads, tokens, head size]
    block = s["block_tables"].long().clamp(min=0)
    length = block.shape[1] * bs
    key, value = s["key_cache"][block], s["value_cache"][block]
    if kv != "auto":
        key, value = key.view(_FP8[kv]), value.view(_FP8[kv])
    key = key.float().permute(0, 2, 1, 4, 3, 5).reshape(b, hk, length, d)
    value = value.float().permute(0, 2, 1, 4, 3).reshape(b, hk, length, d)
    logits = (q @ key.transpose(2, 3)).view(b, hk, widest, group, length) * (s["scale"] * s["k_scale"])
    if case["cap"]:
        logits = case["cap"] * torch.tanh(logits / case["cap"])
    token = torch.arange(length, device=dev)
    drafted = token[None] - ctx[:, None]  # [sequences, tokens]: the place in the tree
    if case["alibi"]:
        pos = s["positions"].long()
        key_pos = torch.where(drafted >= 0, pos[(cu[:-1, None] + drafted.clamp(min=0)).clamp(max=pos.numel() - 1)], token)
        far = (key_pos[:, None] - pos[row][:, :, None]).float()
        logits = logits + s["slopes"].view(1, hk, 1, group, 1) * far[:, None, :, None]
    tree = torch.gather(s["tree_mask"][row], 2, drafted.clamp(0, widest - 1)[:, None].expand(b, widest, length))
    seen = (drafted < 0)[:, None] | (tree & (drafted < count[:, None])[:, None])
    logits = logits.masked_fill(~seen[:, None, :, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isinf(top), 0.0, top))
    del logits
    total = p.sum(-1, keepdim=True)
    p = p.view(b, hk, widest * group, length)
    out = (p @ value).view(b, hk, widest, group, d) / torch.where(total == 0, 1.0, total) * s["v_scale"]
    out = out.permute(0, 2, 1, 3, 4).reshape(b, widest, hk * group, d)
    return out[node[None] < count[:, None]].to(s["query"].dtype)


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_write(state) if op == "write" else _own_read(state) if op == "read" else _own_tree(state)
    return _plain_write(state) if op == "write" else _plain_read(state) if op == "read" else _plain_tree(state)


def work(case):
    lens = _lengths(case)
    hk, d, bs, es, cs = case["kv_heads"], case["head_size"], case["block_size"], _SIZE[case["dtype"]], _cache_bytes(case)
    if case["op"] == "write":
        tokens = len(lens) if case["shape"] == "step" else sum(lens)
        return {"bytes": tokens * 2 * hk * d * (es + cs) + 8 * (tokens + case["pad"]), "flops": 0 if cs == es else 2 * tokens * hk * d}
    if case["op"] == "read":
        tokens = sum(lens)
        pages = sum(-(-(n + case["start"]) // bs) for n in lens)
        return {"bytes": tokens * 2 * hk * d * (es + cs) + 4 * pages + 8 * len(lens), "flops": 0 if cs == es else 2 * tokens * hk * d}
    drafts = _drafts(case)
    h, rows = case["heads"], sum(drafts)
    pages = sum(-(-n // bs) for n in lens)
    return {"bytes": sum(lens) * 2 * hk * d * cs + 2 * rows * h * d * es + rows * case["draft"] + 4 * pages + 8 * len(lens),
            "flops": sum(4 * n * t * h * d for n, t in zip(lens, drafts))}


# ------------------------------------------------------------------------- 64 bits --


def _round_to_8_bits(v, kv):
    """The value of the nearest code of the format (ties to the even one), saturating."""
    mantissa, least = (3, -6) if kv == "fp8_e4m3" else (2, -14)
    top = _FP8_MAX[kv]
    exponent = torch.frexp(v)[1] - 1
    step = torch.pow(2.0, (exponent.clamp(min=least) - mantissa).double())
    return (torch.round(v / step) * step).clamp(-top, top)


def exact(case, seed):
    s = prepare(case, seed)
    kv, hk, d, bs = case["kv"], case["kv_heads"], case["head_size"], case["block_size"]

    def values(cache):
        return (cache if kv == "auto" else cache.view(_FP8[kv])).double()

    if case["op"] == "write":
        k, v = values(s["key_cache"]), values(s["value_cache"])
        slots = s["slots"]
        n = int((slots >= 0).sum())  # padding stands behind the tokens
        key, value = s["key"][:n].double(), s["value"][:n].double()
        if kv != "auto":
            key, value = _round_to_8_bits(key / s["k_scale"], kv), _round_to_8_bits(value / s["v_scale"], kv)
        # one row a slot: [blocks, slots, kv heads, head size]
        flat = k.permute(0, 3, 1, 2, 4).reshape(-1, hk, d)
        flat[slots[:n]] = key
        k = flat.view(k.shape[0], bs, hk, k.shape[2], k.shape[4]).permute(0, 2, 3, 1, 4).contiguous()
        flat = v.permute(0, 3, 1, 2).reshape(-1, hk, d)
        flat[slots[:n]] = value
        return dict(key_cache=k, value_cache=flat.view(v.shape[0], bs, hk, d).permute(0, 2, 3, 1).contiguous())

    def sequence(i, first, last):
        """Keys and values of tokens first..last-1 of sequence i, [kv heads, tokens, head size]."""
        ids = s["block_tables"][i, first // bs:(last - 1) // bs + 1].long()
        cut = slice(first - first // bs * bs, last - first // bs * bs)
        k = values(s["key_cache"][ids]).permute(1, 0, 3, 2, 4).reshape(hk, -1, d)[:, cut] * s["k_scale"]
        v = values(s["value_cache"][ids]).permute(1, 0, 3, 2).reshape(hk, -1, d)[:, cut] * s["v_scale"]
        return k, v

    if case["op"] == "read":
        first = case["start"]
        both = [sequence(i, first, first + n) for i, n in enumerate(_lengths(case))]
        return dict(key=torch.cat([k for k, _ in both], 1).transpose(0, 1).contiguous(),
                    value=torch.cat([v for _, v in both], 1).transpose(0, 1).contiguous())

    lens, drafts, out, at = _lengths(case), _drafts(case), [], 0
    group = case["heads"] // hk
    for i, (n, t) in enumerate(zip(lens, drafts)):
        k, v = sequence(i, 0, n)
        mine = torch.empty(t, hk, group, d, dtype=torch.float64, device=k.device)
        q = s["query"][at:at + t].double().view(t, hk, group, d)
        seen = torch.ones(t, n, dtype=torch.bool, device=k.device)
        seen[:, n - t:] = s["tree_mask"][at:at + t, :t]
        for h in range(hk):
            z = torch.einsum("tgd,nd->tgn", q[:, h], k[h]) * s["scale"]
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if case["alibi"]:
                pos = s["positions"][at:at + t].double()
                where = torch.cat([torch.arange(n - t, device=k.device).double(), pos])
                z = z + s["slopes"].double()[h * group:(h + 1) * group, None] * (where[None, None] - pos[:, None, None])
            z = torch.where(seen[:, None], z, -math.inf)
            mine[:, h] = torch.einsum("tgn,nd->tgd", torch.softmax(z, -1), v[h])
        out.append(mine.view(t, hk * group, d))
        at += t
    return torch.cat(out)
