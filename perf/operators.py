"""Operators over a paged key/value cache kept in the codec's slots, as cases to time and compare.

A page is one slot: ``T`` tokens of one key/value head, ``D`` numbers each (bf16 or fp16), either as it is
(bitmask bit 0) or as the codec's record (bit 1): a participation bit per 32-bit word, then the words, those
that match Bitval under Mask without the masked bits.  The operators:

  pages   copying, forking, freeing and compacting pages;
  bounds  the smallest and the largest key of a page, number by number: a page's cheap summary;
  sparse  per query and head, the pages with the highest bound on the score, and attention over those;
  tree    attention of a tree of drafted tokens over the cached pages and over the drafted ancestors.

``own`` False: plain torch, 32 bits (the page scores in 64, since neighbouring scores decide which pages are
read).  ``own`` True: the package's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    """The cases.  heads/head_dim/page_tokens follow the repository's KV workload (32 heads, 128 dims, 16-token
    pages of 4 KiB); `kv_heads` below `heads` are grouped queries; `period` is the Mask period in bits: a whole
    page as in that workload, or one token's row."""
    kv = dict(heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", period=2048, packed=True)
    return [
        # the step that decodes one token of one chat: nothing but latency
        dict(kv, name="tree_one_token", op="tree", seqs=1, ctx=1000, new=1, ragged=False),
        # speculative decoding of eight streams with up to 24 drafted tokens each, ragged contexts
        dict(kv, name="tree_eight_streams", op="tree", seqs=8, ctx=8200, new=24, ragged=True),
        # two long documents, 64 drafted tokens, pages not compressed: the largest attention
        dict(kv, name="tree_long_documents", op="tree", seqs=2, ctx=65521, new=64, ragged=False, heads=64,
             dtype="fp16", packed=False),
        # a narrow model's batch, 64 dims, 32-token pages, the whole-page Mask period
        dict(kv, name="tree_narrow_heads", op="tree", seqs=16, ctx=4096, new=7, ragged=True, heads=16, kv_heads=16,
             dim=64, page=32, period=32768),
        # one token that reads 16 of its 256 pages
        dict(kv, name="sparse_one_token", op="sparse", seqs=1, rows=1, ctx=4090, top=16, ragged=False),
        # a decoding batch over 32 K tokens each, 64 pages of 2,048 per head
        dict(kv, name="sparse_decode_batch", op="sparse", seqs=16, rows=16, ctx=32768, top=64, ragged=True),
        # a block of 512 prompt tokens of one 64 K document, 128 pages for each
        dict(kv, name="sparse_prompt_block", op="sparse", seqs=1, rows=512, ctx=65536, top=128, ragged=False,
             dtype="fp16", packed=False),
        # the pages that one decoding step of 64 streams has filled
        dict(kv, name="bounds_step", op="bounds", pages=67, slots=4096),
        # the whole cache of a prompt, under the repository's KV format
        dict(kv, name="bounds_prompt", op="bounds", pages=65536, slots=65536, period=32768),
        # a stream's pages brought back into the pool
        dict(kv, name="pages_copy_stream", op="copy", pages=263, slots=2048),
        # beams forked off their parents and dropped again
        dict(kv, name="pages_fork_beams", op="fork", seqs=12, forks=12, ctx=4100, slots=32768),
        # a pool of 256 MiB that has become half empty
        dict(kv, name="pages_compact_pool", op="compact", slots=65536, live=0.55),
    ]


def draw(rng):
    def logint(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    dim, page = rng.choice([(128, 16), (128, 16), (128, 32), (64, 16), (64, 32), (64, 64)])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(heads=kv_heads * rng.choice([1, 2, 4, 7, 8]), kv_heads=kv_heads, dim=dim, page=page,
             dtype=rng.choice(["bf16", "fp16"]), period=rng.choice([32, dim * 16, page * dim * 16]),
             packed=rng.random() < 0.7)
    op = rng.choice(["tree", "tree", "sparse", "sparse", "bounds", "copy", "fork", "compact"])
    c["op"] = op
    if op == "tree":
        c.update(seqs=logint(1, 8), ctx=logint(1, 16384), new=logint(1, 64), ragged=rng.random() < 0.6)
    elif op == "sparse":
        seqs = logint(1, 8)
        c.update(seqs=seqs, rows=seqs * logint(1, 24), ctx=logint(1, 32768), top=logint(4, 96),
                 ragged=rng.random() < 0.6)
    elif op in ("bounds", "copy"):
        c["pages"] = logint(1, 32768)
        c["slots"] = c["pages"] * (1 if op == "bounds" else 2) + rng.randrange(70)
    elif op == "fork":
        c.update(seqs=logint(1, 16), ctx=logint(1, 4096))
        c["forks"] = c["seqs"]
        c["slots"] = _fork_slots(c) + rng.randrange(5000)
    else:
        c.update(slots=logint(40, 40000), live=rng.uniform(0.05, 0.95))
    return c


# --- sizes that follow from a case alone -------------------------------------------------------------------


def _page_bytes(c):
    return c["page"] * c["dim"] * 2


def _blocks(c):
    return -(-c["ctx"] // c["page"])


def _seq_lens(c):
    """Context tokens of each sequence: the first has all of them, ragged ones between a third and all."""
    share = 0.35 + 0.65 * ((np.arange(c["seqs"]) * 0.618) % 1.0)
    share[0] = 1.0
    lens = np.maximum(1, (c["ctx"] * (share if c.get("ragged") else np.ones(c["seqs"]))).astype(np.int64))
    return lens


def _new_counts(c):
    """Drafted tokens of each sequence."""
    if not c["ragged"]:
        return np.full(c["seqs"], c["new"], np.int64)
    return 1 + (np.arange(c["seqs"]) * 5 + c["new"] - 1) % c["new"]


def _row_lens(c):
    """Context tokens that each query of a sparse case sees: its sequence's, the rows of one sequence being
    consecutive tokens of it."""
    per = c["rows"] // c["seqs"]
    back = np.arange(per)[::-1]
    return np.maximum(1, _seq_lens(c)[:, None] - back[None, :]).reshape(-1)


def _fork_slots(c):
    blocks = int((-(-_seq_lens(c) // c["page"])).sum())
    return c["kv_heads"] * (blocks + c["forks"])


def work(case):
    c, L, e = case, _page_bytes(case), 2
    if c["op"] == "tree":
        blocks = int((-(-_seq_lens(c) // c["page"])).sum())
        n = _new_counts(c)
        rows = int(n.sum())
        pairs = int((_seq_lens(c) * n).sum()) + int((n * n).sum()) // 2
        return {"bytes": 2 * blocks * c["kv_heads"] * L + 2 * rows * c["heads"] * c["dim"] * e
                + 2 * rows * c["kv_heads"] * c["dim"] * e + 4 * rows * c["heads"],
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "sparse":
        lens = _row_lens(c)
        blocks = -(-lens // c["page"])
        # summaries and pages that several queries share are counted once per sequence
        per = c["rows"] // c["seqs"]
        seq_blocks = -(-_seq_lens(c) // c["page"])
        picked = np.minimum(blocks, c["top"])
        pages = np.minimum(picked.reshape(c["seqs"], per).sum(1), seq_blocks).sum()
        return {"bytes": int(seq_blocks.sum()) * c["kv_heads"] * 2 * c["dim"] * e + 2 * int(pages) * c["kv_heads"] * L
                + c["rows"] * c["heads"] * (2 * c["dim"] * e + 4) + c["rows"] * c["kv_heads"] * c["top"] * 4,
                "flops": int(blocks.sum()) * c["heads"] * c["dim"] * 4
                + int(picked.sum()) * c["page"] * c["heads"] * c["dim"] * 4}
    if c["op"] == "bounds":
        return {"bytes": c["pages"] * (L + 2 * c["dim"] * e + 12), "flops": 2 * c["pages"] * c["page"] * c["dim"]}
    if c["op"] == "copy":
        return {"bytes": c["pages"] * (2 * L + 16), "flops": 0}
    if c["op"] == "fork":
        entries = 2 * c["kv_heads"] * c["forks"] * _blocks(c)
        return {"bytes": entries * 16 + 2 * c["kv_heads"] * c["forks"] * L + 4 * c["slots"], "flops": 0}
    moved = int(c["slots"] * c["live"] * (1 - c["live"]))
    return {"bytes": 2 * moved * L + 24 * c["slots"], "flops": 0}


# --- inputs ------------------------------------------------------------------------------------------------


def _values(c, n, g, spread=1.0):
    """n pages of N(0, 1) times a scale per dim, drawn from lognormal(0, 1) as in the repository's KV workload;
    a page of a head keeps its head's scales."""
    scale = torch.empty(c["kv_heads"], 1, c["dim"], device="cuda").log_normal_(0.0, spread, generator=g)
    x = torch.randn(n, c["page"], c["dim"], device="cuda", generator=g)
    x *= scale[torch.arange(n, device="cuda") % c["kv_heads"]]
    return x.to(DTYPES[c["dtype"]])


def _metadata(words, period_words):
    """Mask and Bitval of a sample: the bits on which 95 % of the sample's periods agree."""
    sample = words[:1024].reshape(-1, period_words)
    n = sample.shape[0]
    bit = torch.arange(32, device=words.device, dtype=torch.int32)
    ones = ((sample.unsqueeze(-1) >> bit) & 1).sum(0)
    need = math.ceil(0.95 * n)
    m = torch.maximum(ones, n - ones) >= need
    v = m & (2 * ones > n)
    weight = torch.ones(32, dtype=torch.int64, device=words.device) << bit.long()
    return ((t.long() * weight).sum(-1) for t in (m, v))


def _moves(mask):
    """For each word of Mask, which of its kept bits move by 1, 2, 4, 8 and 16 places (one row for each distance)
    when they are brought together at the low end: a bit moves by the number of masked bits below it."""
    bit = torch.arange(32, device=mask.device)
    keep = ((mask[:, None] >> bit) & 1) ^ 1
    far = (1 - keep).cumsum(1) * keep
    rows = []
    for i in range(5):
        at = bit - (far & ((1 << i) - 1))  # where the shorter moves have put the bit
        rows.append((((far >> i) & 1) << at).sum(1))
    return torch.stack(rows)


def _store(words, mask, bitval, moves):
    """The slots (int32 words) and bitmask bits (bool) of pages given as int32 words."""
    n, nw = words.shape
    hw = (nw + 31) // 32
    slots, bits = torch.empty_like(words), torch.empty(n, dtype=torch.bool, device=words.device)
    m, b = mask.repeat(nw // mask.numel()), bitval.repeat(nw // mask.numel())
    moves = moves.repeat(1, nw // mask.numel())
    width = 32 - ((m.unsqueeze(-1) >> torch.arange(32, device=m.device)) & 1).sum(-1)
    step = max(1, (1 << 26) // nw)
    for a in range(0, n, step):
        x = words[a:a + step].long() & 0xFFFFFFFF
        p = (x & m) == b
        field = x & ~m
        for i in range(5):
            t = field & moves[i]
            field = (field ^ t) | (t >> (1 << i))
        field = torch.where(p, field, x)
        size = torch.where(p, width.expand_as(x), torch.full_like(x, 32))
        end = size.cumsum(1)
        at = end - size + 32 * hw
        total = (end[:, -1] + 32 * hw + 31) // 32
        rec = torch.zeros(x.shape[0], nw + hw + 2, dtype=torch.int64, device=x.device)
        low = (field << (at & 31)) & 0xFFFFFFFF
        rec.scatter_add_(1, at >> 5, low)
        rec.scatter_add_(1, (at >> 5) + 1, (field >> (32 - (at & 31))))
        w32 = torch.nn.functional.pad(p, (0, hw * 32 - nw)).reshape(-1, hw, 32).long()
        rec[:, :hw] = (w32 << torch.arange(32, device=x.device)).sum(-1)
        ok = total < nw
        out = torch.where(ok[:, None], rec[:, :nw], x)
        slots[a:a + step] = torch.where(out >= 1 << 31, out - (1 << 32), out).int()
        bits[a:a + step] = ok
    return slots, bits


def _pack_bits(bits):
    n = bits.numel()
    w = torch.nn.functional.pad(bits, (0, -n % 32)).reshape(-1, 32).long()
    w = (w << torch.arange(32, device=bits.device)).sum(1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def _pool(c, values):
    """A pool of pages: slots, bitmask and the metadata they were stored with, and the codec's handle."""
    n = values.shape[0]
    words = values.reshape(n, -1).view(torch.int32)
    mask, bitval = _metadata(words, c["period"] // 32)
    moves = _moves(mask)
    if c["packed"]:
        slots, bits = _store(words, mask, bitval, moves)
    else:
        slots, bits = words.clone(), torch.zeros(n, dtype=torch.bool, device="cuda")
    pool = {"slots": slots, "bitmask": _pack_bits(bits), "mask": mask, "bitval": bitval, "moves": moves, "n": n}
    if own:  # the handle, which a program keeps for as long as the pool
        from lossless_tensor_compression_ibp_amd import ibp
        pool["meta"] = ibp.ibp_meta_create(_page_bytes(c), 32, c["period"], mask.cpu().numpy().astype(np.uint32),
                                           bitval.cpu().numpy().astype(np.uint32))
        pool["pages"] = ibp.Pages(pool["meta"], slots, n, pool["bitmask"])
    return pool


def _tables(c, lens, n_slots, g, extra=0):
    """Page ids (sequences, kv heads, blocks), -1 past a sequence's last block; the pages lie scattered."""
    blocks = torch.from_numpy(-(-lens // c["page"])).cuda()
    most = int(blocks.max())
    live = torch.arange(most, device="cuda")[None, :] < blocks[:, None]
    live = live[:, None, :].expand(-1, c["kv_heads"], -1)
    rank = live.reshape(-1).long().cumsum(0) - 1
    order = torch.randperm(n_slots, device="cuda", generator=g)
    t = torch.where(live.reshape(-1), order[rank.clamp(min=0)], torch.full_like(rank, -1))
    return t.reshape(len(lens), c["kv_heads"], most).contiguous()


def _cache(c, lens, seed, g):
    n = c["kv_heads"] * int((-(-lens // c["page"])).sum()) + 37
    st = {"c": c}
    kx, vx = _values(c, n, g), _values(c, n, g, 0.5)
    st["k"], st["v"] = _pool(c, kx), _pool(c, vx)
    st["k_table"], st["v_table"] = _tables(c, lens, n, g), _tables(c, lens, n, g)
    return st, kx, vx


def _inputs(case, seed):
    """The state, and the pages' values as they were before they were stored."""
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))
    rs = np.random.RandomState(seed % (1 << 31))
    dt = DTYPES[c["dtype"]]
    T, D, H, HK = c["page"], c["dim"], c["heads"], c["kv_heads"]

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g).to(dt)

    if c["op"] == "tree":
        lens, n = _seq_lens(c), _new_counts(c)
        st, kx, vx = _cache(c, lens, seed, g)
        rows = int(n.sum())
        st.update(lens=torch.from_numpy(lens).int().cuda(), max_len=int(lens.max()), max_new=int(n.max()),
                  new_rows=torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).int().cuda(),
                  q=rand(rows, H, D), k_new=rand(rows, HK, D), v_new=rand(rows, HK, D))
        mask = np.zeros((rows, 1), np.uint64)
        r = 0
        for m in n:  # each drafted token sees itself and its ancestors
            seen = []
            for i in range(int(m)):
                parent = rs.randint(-1, i) if i else -1
                seen.append((1 << i) | (seen[parent] if parent >= 0 else 0))
                mask[r + i, 0] = seen[-1]
            r += int(m)
        st["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
        return st, kx, vx
    if c["op"] == "sparse":
        lens = _row_lens(c)
        st, kx, vx = _cache(c, _seq_lens(c), seed, g)
        per = c["rows"] // c["seqs"]
        st.update(lens=torch.from_numpy(lens).int().cuda(), q=rand(c["rows"], H, D),
                  row_seq=torch.arange(c["rows"], device="cuda", dtype=torch.int32) // per, max_len=int(lens.max()),
                  bounds=torch.stack([kx.amin(1), kx.amax(1)], 1).contiguous())
        return st, kx, vx
    if c["op"] == "bounds":
        kx = _values(c, c["slots"], g)
        ids = torch.randperm(c["slots"], device="cuda", generator=g)[:c["pages"]].contiguous()
        tokens = torch.full((c["pages"],), T, dtype=torch.int32, device="cuda")
        tokens[::7] = 1 + torch.arange(tokens[::7].numel(), device="cuda", dtype=torch.int32) % T
        return {"c": c, "k": _pool(c, kx), "ids": ids, "tokens": tokens,
                "bounds": torch.zeros(c["slots"], 2, D, dtype=dt, device="cuda")}, kx, None
    kx = _values(c, c["slots"], g)
    st = {"c": c, "k": _pool(c, kx)}
    if c["op"] == "copy":
        st["to"] = {"slots": torch.zeros_like(st["k"]["slots"]), "n": c["slots"],
                    "bitmask": torch.zeros_like(st["k"]["bitmask"])}
        st["src"] = torch.randperm(c["slots"], device="cuda", generator=g)[:c["pages"]].contiguous()
        st["dst"] = torch.randperm(c["slots"], device="cuda", generator=g)[:c["pages"]].contiguous()
    elif c["op"] == "fork":
        lens = _seq_lens(c)
        t = _tables(c, lens, c["slots"], g)
        st["refs"] = torch.zeros(c["slots"], dtype=torch.int32, device="cuda")
        st["refs"][t[t >= 0]] = 1
        st["table"] = torch.cat([t, torch.full((c["forks"],) + tuple(t.shape[1:]), -1, device="cuda")]).contiguous()
        st["lens"] = torch.from_numpy(np.concatenate([lens, np.zeros(c["forks"], np.int64)])).int().cuda()
        st["parents"] = torch.from_numpy(rs.randint(0, c["seqs"], c["forks"])).cuda()
        st["children"] = c["seqs"] + torch.randperm(c["forks"], device="cuda", generator=g)
    else:
        live = torch.randperm(c["slots"], device="cuda", generator=g) < round(c["slots"] * c["live"])
        refs = live.int() * (1 + torch.arange(c["slots"], device="cuda", dtype=torch.int32) % 3)
        ids = torch.nonzero(live)[:, 0]
        table = torch.cat([ids[torch.randperm(ids.numel(), device="cuda", generator=g)],
                           torch.full((17,), -1, device="cuda")])
        st.update(refs0=refs, table0=table, bitmask0=st["k"]["bitmask"].clone(), refs=refs.clone(),
                  table=table.clone(), map=torch.empty(c["slots"], dtype=torch.int64, device="cuda"),
                  n_live=torch.empty(1, dtype=torch.int64, device="cuda"))
    return st, kx, None


def prepare(case, seed):
    return _inputs(case, seed)[0]


# --- the plain forms ---------------------------------------------------------------------------------------


def _bit_of(bitmask, ids):
    return ((bitmask[ids >> 5] >> (ids & 31).int()) & 1).bool()


def _widths(c, pool):
    """Bits that a matching word keeps, word by word of a page."""
    nw = _page_bytes(c) // 4
    m = pool["mask"].repeat(nw // pool["mask"].numel())
    return m, 32 - ((m.unsqueeze(-1) >> torch.arange(32, device=m.device)) & 1).sum(-1)


def _participation(slots, nw):
    hw = (nw + 31) // 32
    h = slots[:, :hw].long()
    return ((h.unsqueeze(-1) >> torch.arange(32, device=h.device)) & 1).reshape(h.shape[0], -1)[:, :nw].bool()


def _load(c, pool, ids):
    """The values (pages, page tokens, dim) of the pages `ids`, decoded where they hold a record."""
    words = pool["slots"][ids]
    if c["packed"]:
        n, nw = words.shape
        hw = (nw + 31) // 32
        m, width = _widths(c, pool)
        b = pool["bitval"].repeat(nw // pool["bitval"].numel())
        comp = _bit_of(pool["bitmask"], ids)[:, None]
        p = _participation(words, nw)
        size = torch.where(p, width, torch.full_like(width, 32))
        at = size.cumsum(1) - size + 32 * hw
        w = words.long() & 0xFFFFFFFF
        low = at >> 5
        f = w.gather(1, low.clamp(max=nw - 1)) | (w.gather(1, (low + 1).clamp(max=nw - 1)) << 32)
        f = (f >> (at & 31)) & 0xFFFFFFFF
        x, moves = f, pool["moves"].repeat(1, nw // pool["mask"].numel())
        for i in (4, 3, 2, 1, 0):  # the kept bits back to their places, the farthest moves first
            back = moves[i] >> (1 << i)
            x = (x & ~(moves[i] | back)) | ((x & back) << (1 << i))
        x = torch.where(comp, torch.where(p, (x & ~m) | b, f), w)
        words = torch.where(x >= 1 << 31, x - (1 << 32), x).int()
    return words.contiguous().view(DTYPES[c["dtype"]]).reshape(ids.numel(), c["page"], c["dim"])


def _softmax_over(s, seen):
    """Weights and log-sum-exp of the scores `s` where `seen`; rows that see nothing weigh nothing."""
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total), (top + torch.log(total))[..., 0]


def _context(st, table, pool):
    """(sequences, kv heads, tokens, dim) in 32 bits; what lies past a sequence's end is zero or stale."""
    c = st["c"]
    b, h, n = table.shape
    return _load(c, pool, table.clamp(min=0).reshape(-1)).reshape(b, h, n * c["page"], c["dim"]).float()


def _plain_tree(st):
    c = st["c"]
    G, most = c["heads"] // c["kv_heads"], st["max_new"]
    k, v = _context(st, st["k_table"], st["k"]), _context(st, st["v_table"], st["v"])
    first, count = st["new_rows"][:-1].long(), (st["new_rows"][1:] - st["new_rows"][:-1]).long()
    slot = torch.arange(most, device="cuda")
    held = slot[None, :] < count[:, None]
    row = (first[:, None] + slot[None, :]).clamp(max=st["q"].shape[0] - 1)  # (sequences, drafted)

    def of_heads(x, groups):
        x = x.float()[row]  # (seqs, drafted, heads, dim)
        return x.reshape(c["seqs"], most, c["kv_heads"], groups, c["dim"]).permute(0, 2, 1, 3, 4)

    q = of_heads(st["q"], G).reshape(c["seqs"], c["kv_heads"], most * G, c["dim"])
    k = torch.cat([k, of_heads(st["k_new"], 1)[:, :, :, 0]], 2)
    v = torch.cat([v, of_heads(st["v_new"], 1)[:, :, :, 0] * held[:, None, :, None]], 2)
    ctx = k.shape[2] - most
    seen = (torch.arange(ctx, device="cuda")[None, :] < st["lens"][:, None])[:, None, :].expand(-1, most, -1)
    tree = ((st["mask"][row][..., 0][..., None] >> slot) & 1).bool() & held[:, None, :]
    seen = torch.cat([seen, tree], 2)  # (seqs, drafted, tokens)
    s = torch.matmul(q, k.transpose(2, 3)) * (c["dim"] ** -0.5)
    p, lse = _softmax_over(s, seen[:, None].repeat_interleave(G, 2))
    o = torch.matmul(p, v).reshape(c["seqs"], c["kv_heads"], most, G, c["dim"]).permute(0, 2, 1, 3, 4)
    lse = lse.reshape(c["seqs"], c["kv_heads"], most, G).permute(0, 2, 1, 3)
    # back to the ragged rows
    owner = torch.searchsorted(st["new_rows"][1:].contiguous(),
                               torch.arange(st["q"].shape[0], device="cuda", dtype=torch.int32), right=True)
    place = torch.arange(st["q"].shape[0], device="cuda") - first[owner]
    o = o[owner, place].reshape(-1, c["heads"], c["dim"])
    return o.to(st["q"].dtype), lse[owner, place].reshape(-1, c["heads"]).contiguous()


def _plain_select(st):
    """Per query and kv head the `top` pages: the first, the last two, then those with the highest bound
    max over the group's heads of sum over dims of max(q lo, q hi); ascending, -1 behind."""
    c = st["c"]
    HK, G, D, top = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["top"]
    table = st["k_table"]
    B, n = table.shape[0], table.shape[2]
    bounds = st["bounds"][table.clamp(min=0)].double()  # (seqs, kv heads, blocks, 2, dim)
    per = c["rows"] // c["seqs"]
    q = st["q"].double().reshape(B, per, HK, G, D).permute(0, 2, 1, 3, 4).reshape(B, HK, per * G, D)
    s = torch.matmul(q.clamp(min=0), bounds[..., 1, :].transpose(2, 3)) \
        + torch.matmul(q.clamp(max=0), bounds[..., 0, :].transpose(2, 3))
    s = s.reshape(B, HK, per, G, n).amax(3).float().permute(0, 2, 1, 3).reshape(c["rows"], HK, n)
    block = torch.arange(n, device="cuda")
    blocks = ((st["lens"] + c["page"] - 1) // c["page"])[:, None, None]
    s = torch.where((block < 1) | (block >= blocks - 2), torch.full_like(s, math.inf), s)
    s = torch.where(block < blocks, s, torch.full_like(s, -math.inf))
    order = torch.sort(s, dim=-1, descending=True, stable=True)[1][..., :top]
    order = torch.where(order < blocks, order, torch.full_like(order, 1 << 30)).sort(-1)[0]
    order = torch.where(order == 1 << 30, torch.full_like(order, -1), order).int()
    return torch.nn.functional.pad(order, (0, top - order.shape[-1]), value=-1).contiguous()


def _plain_sparse(st):
    c = st["c"]
    HK, G, D, T = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["page"]
    blocks = _plain_select(st)
    seq = st["row_seq"].long()[:, None, None]
    head = torch.arange(HK, device="cuda")[None, :, None]
    at = blocks.clamp(min=0).long()
    k, v = (_load(c, st[n], st[n + "_table"][seq, head, at].clamp(min=0).reshape(-1)).float()
            .reshape(c["rows"], HK, -1, D) for n in "kv")
    token = at[..., None] * T + torch.arange(T, device="cuda")
    seen = ((blocks >= 0)[..., None] & (token < st["lens"][:, None, None, None])).reshape(c["rows"], HK, 1, -1)
    q = st["q"].float().reshape(c["rows"], HK, G, D)
    s = torch.matmul(q, k.transpose(2, 3)) * (D ** -0.5)
    p, lse = _softmax_over(s, seen)
    o = torch.matmul(p, v).reshape(c["rows"], c["heads"], D)
    return blocks, o.to(st["q"].dtype), lse.reshape(c["rows"], c["heads"])


def _plain_bounds(st):
    c = st["c"]
    x = _load(c, st["k"], st["ids"]).float()
    held = (torch.arange(c["page"], device="cuda")[None, :] < st["tokens"][:, None])[:, :, None]
    st["bounds"][st["ids"], 0] = x.masked_fill(~held, math.inf).amin(1).to(st["bounds"].dtype)
    st["bounds"][st["ids"], 1] = x.masked_fill(~held, -math.inf).amax(1).to(st["bounds"].dtype)
    return st["bounds"]


def _set_bits(bitmask, ids, bits):
    """The bits `ids` of the mask set to `bits`, the others left."""
    n = bitmask.numel() * 32
    every = ((bitmask[:, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).reshape(n).bool()
    every[ids] = bits
    bitmask.copy_(_pack_bits(every))


def _plain_copy(c, pool, src, to, dst):
    """Pages src of the pool into slots dst: a record's words, or the whole page; what lies behind stays."""
    x = pool["slots"][src]
    bits = _bit_of(pool["bitmask"], src)
    nw = x.shape[1]
    _, width = _widths(c, pool)
    size = torch.where(_participation(x, nw), width, torch.full_like(width, 32)).sum(1)
    words = torch.where(bits, (nw + 31) // 32 + (size + 31) // 32, torch.full_like(size, nw))
    keep = torch.arange(nw, device="cuda")[None, :] < words[:, None]
    to["slots"][dst] = torch.where(keep, x, to["slots"][dst])
    _set_bits(to["bitmask"], dst, bits)


def _plain_fork(st):
    c, table, refs = st["c"], st["table"], st["refs"]
    T, n = c["page"], st["table"].shape[2]
    lens = st["lens"][st["parents"]].long()
    full = (torch.arange(n, device="cuda")[None, :] < (lens // T)[:, None])[:, None, :]  # shared pages
    rows = table[st["parents"]]
    shared = torch.where(full, rows, torch.full_like(rows, -1))
    refs.index_add_(0, shared.clamp(min=0).reshape(-1), (shared >= 0).reshape(-1).int())
    # the page that is still being filled is copied, into the lowest free slots in order
    tail = (lens % T != 0)[:, None].expand(-1, c["kv_heads"]).reshape(-1)
    rank = tail.long().cumsum(0) - 1
    free = torch.sort((refs != 0).int(), stable=True)[1]
    at = torch.nonzero(tail)[:, 0]
    new = free[rank[at]]
    refs[new] = 1
    old = rows.gather(2, (lens // T).clamp(max=n - 1)[:, None, None].expand(-1, c["kv_heads"], 1)).reshape(-1)[at]
    _plain_copy(c, st["k"], old, st["k"], new)
    child = shared.reshape(-1, n)
    child[at, (lens // T).repeat_interleave(c["kv_heads"])[at]] = new
    table[st["children"]] = child.reshape(rows.shape)
    after = (table[st["children"]].clone(), refs.clone())
    gone = table[st["children"]].reshape(-1)
    refs.index_add_(0, gone.clamp(min=0), -(gone >= 0).int())
    table[st["children"]] = -1
    return after + (refs, table, st["k"]["slots"], st["k"]["bitmask"])


def _plain_compact(st):
    """The last live page moves to the first hole, and so on, until the live pages lie in front."""
    c, pool = st["c"], st["k"]
    live = st["refs"] > 0
    at = torch.arange(c["slots"], device="cuda")
    n_live = live.long().sum()
    holes = torch.nonzero(~live & (at < n_live))[:, 0]
    movers = torch.nonzero(live & (at >= n_live))[:, 0].flip(0)
    _plain_copy(c, pool, movers, pool, holes)
    st["map"].copy_(torch.where(live, at, torch.full_like(at, -1)))
    st["map"][movers] = holes
    st["refs"][holes] = st["refs"][movers]
    st["refs"][movers] = 0
    st["table"].copy_(torch.where(st["table"] >= 0, st["map"][st["table"].clamp(min=0)], st["table"]))
    st["n_live"].copy_(n_live)


# --- one pass ----------------------------------------------------------------------------------------------


def run(state):
    st, c = state, state["c"]
    if own:
        from lossless_tensor_compression_ibp_amd import ibp
    if c["op"] == "tree":
        if not own:
            return _plain_tree(st)
        out = torch.empty_like(st["q"])
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
        ibp.ibp_tree_attention(st["k"]["pages"], st["v"]["pages"], st["q"], st["k_table"], st["v_table"], st["lens"],
                               st["new_rows"], st["k_new"], st["v_new"], st["mask"], out, lse,
                               scale=c["dim"] ** -0.5, max_len=st["max_len"], max_new=st["max_new"])
        return out, lse
    if c["op"] == "sparse":
        if not own:
            return _plain_sparse(st)
        blocks = torch.empty(c["rows"], c["kv_heads"], c["top"], dtype=torch.int32, device="cuda")
        out = torch.empty_like(st["q"])
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
        ibp.ibp_select_pages(st["q"], st["bounds"], st["k_table"], st["lens"], blocks, meta=st["k"]["meta"],
                             page_tokens=c["page"], keep_first=1, keep_last=2, row_seq=st["row_seq"])
        ibp.ibp_sparse_attention(st["k"]["pages"], st["v"]["pages"], st["q"], st["k_table"], st["v_table"],
                                 st["lens"], blocks, out, lse, scale=c["dim"] ** -0.5, row_seq=st["row_seq"])
        return blocks, out, lse
    if c["op"] == "bounds":
        if not own:
            return _plain_bounds(st)
        ibp.ibp_page_bounds(st["k"]["pages"], st["ids"], st["tokens"], st["bounds"])
        return st["bounds"]
    if c["op"] == "copy":
        if own:
            ibp.ibp_pages_copy(st["k"]["meta"], st["k"]["slots"], st["k"]["n"], st["k"]["bitmask"], st["src"],
                               st["to"]["slots"], st["to"]["n"], st["to"]["bitmask"], st["dst"])
        else:
            _plain_copy(c, st["k"], st["src"], st["to"], st["dst"])
        return st["to"]["slots"], st["to"]["bitmask"]
    if c["op"] == "fork":
        if not own:
            return _plain_fork(st)
        pool = st["k"]
        ibp.ibp_pages_fork(pool["meta"], pool["slots"], pool["n"], pool["bitmask"], st["refs"], st["table"], st["lens"],
                           st["parents"], st["children"], page_tokens=c["page"])
        after = (st["table"][st["children"]], st["refs"].clone())
        ibp.ibp_pages_free(pool["meta"], st["refs"], pool["n"], st["table"], st["children"])
        return after + (st["refs"], st["table"], pool["slots"], pool["bitmask"])
    # compaction: the pool as it was before the first pass, whose pages still lie where they were
    st["refs"].copy_(st["refs0"])
    st["table"].copy_(st["table0"])
    st["k"]["bitmask"].copy_(st["bitmask0"])
    if own:
        pool = st["k"]
        ibp.ibp_pages_compact(pool["meta"], pool["slots"], pool["n"], pool["bitmask"], st["refs"], st["map"],
                              st["n_live"], table=st["table"])
    else:
        _plain_compact(st)
    return st["map"], st["refs"], st["table"], st["n_live"], st["k"]["slots"], st["k"]["bitmask"]


# --- in 64 bits, from the definition -----------------------------------------------------------------------


def _attend(q, k, v, seen):
    """One head group: q (rows, dim), k and v (tokens, dim), seen (rows, tokens)."""
    s = (q.double() @ k.double().T) / math.sqrt(q.shape[1])
    s[~seen] = -math.inf
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return p @ v.double(), lse


def _chosen(q, lo, hi, n, top):
    """The blocks that one query's heads q (heads, dim) read of its n blocks with bounds lo and hi."""
    s = torch.maximum(q.double()[:, None] * lo.double(), q.double()[:, None] * hi.double()).sum(2).amax(0).float()
    s = s.cpu().numpy()[:n]
    forced = np.zeros(n, bool)
    forced[:1] = forced[-2:] = True
    best = np.lexsort((np.arange(n), -s, ~forced))[:top]
    return torch.from_numpy(np.sort(best)).cuda()


def exact(case, seed):
    c = dict(case)
    if c["op"] not in ("tree", "sparse", "bounds"):
        return None  # pages are moved and compared, not computed
    st, kx, vx = _inputs(case, seed)
    if c["op"] == "bounds":
        r = torch.zeros_like(st["bounds"], dtype=torch.float64)
        held = torch.arange(c["page"], device="cuda")[:, None] < st["tokens"][:, None, None]
        x = kx[st["ids"]].double()
        r[st["ids"], 0] = torch.where(held, x, x[:, :1]).min(1)[0]
        r[st["ids"], 1] = torch.where(held, x, x[:, :1]).max(1)[0]
        return r
    T, D, HK, G = c["page"], c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    rows = st["q"].shape[0]
    out = torch.zeros(rows, c["heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, c["heads"], dtype=torch.float64, device="cuda")
    if c["op"] == "tree":
        ends, lens = st["new_rows"].tolist(), st["lens"].tolist()
        for b in range(c["seqs"]):
            lo, hi = ends[b], ends[b + 1]
            n = hi - lo
            seen = torch.ones(n, lens[b] + n, dtype=torch.bool, device="cuda")
            seen[:, lens[b]:] = ((st["mask"][lo:hi] >> torch.arange(n, device="cuda")) & 1).bool()
            nb = -(-lens[b] // T)
            for h in range(HK):
                k = torch.cat([kx[st["k_table"][b, h, :nb]].reshape(-1, D)[:lens[b]], st["k_new"][lo:hi, h]])
                v = torch.cat([vx[st["v_table"][b, h, :nb]].reshape(-1, D)[:lens[b]], st["v_new"][lo:hi, h]])
                for i in range(h * G, h * G + G):
                    out[lo:hi, i], lse[lo:hi, i] = _attend(st["q"][lo:hi, i], k, v, seen)
        return out, lse
    if rows * HK > 6000:
        return None
    lens, seq = st["lens"].tolist(), st["row_seq"].tolist()
    for r in range(rows):
        for h in range(HK):
            table = st["k_table"][seq[r], h]
            lo, hi = st["bounds"][table.clamp(min=0)].unbind(1)
            b = _chosen(st["q"][r, h * G:(h + 1) * G], lo, hi, -(-lens[r] // T), c["top"])
            at = (b[:, None] * T + torch.arange(T, device="cuda")).reshape(-1)
            k = kx[st["k_table"][seq[r], h, b]].reshape(-1, D)
            v = vx[st["v_table"][seq[r], h, b]].reshape(-1, D)
            see = (at < lens[r])[None, :].expand(G, -1)
            out[r, h * G:(h + 1) * G], lse[r, h * G:(h + 1) * G] = _attend(st["q"][r, h * G:(h + 1) * G], k, v, see)
    return None, out, lse
