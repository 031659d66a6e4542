"""Cases, plain forms and exact results of the serving operators around the paged latent cache.

Three operators, over the cache that the decode step reads:

* ``prompt``: attention of the query tokens of packed sequences (whole prompts, or the last
  chunk of a longer context) over each sequence's own cached rows, causal, with the latent
  blocks' head groups; ``mlra_prefill``.
* ``shared``: one decode step of a batch whose sequences share long prefixes in groups, each
  prefix attended to once for all its members; ``mlra_decode_prefix``.
* ``fork`` / ``compact`` / ``turn``: the pages of the cache: forking sequences onto shared
  pages, moving the used pages to the front of the pool, and a scheduler's turn (free finished
  sequences, reserve pages for growing ones, fork); ``mlra_fork_pages``,
  ``mlra_compact_pages``, ``mlra_free_pages``, ``mlra_reserve_pages``.

With ``own`` false ``run`` computes the operators in elementary torch operations in 32 bits;
with ``own`` true it calls the library. ``exact`` computes them in 64 bits from the
un-absorbed definition (each head's keys and values formed from the cached latent).
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
# (k, h, d_h, d_c, d_rope): the layer shapes of the decode workloads
SHAPES = {
    "mlra4": (4, 128, 128, 512, 64),
    "mlra2": (2, 128, 128, 512, 64),
    "mla": (1, 128, 128, 512, 64),
    "rank4": (1, 32, 128, 128, 64),      # one MLRA-4 rank of 4-way tensor parallelism
}
E4M3_SCALE = 2.0 ** -5                   # value of a cached E4M3 byte = E4M3_SCALE * e4m3(byte)
MAX_PAIRS = 16384 * 16385 // 2 * 128     # (query, key, head) triples of the largest listed prompt


def listed():
    return [
        # ---- attention over prompts ----
        # verification of a few drafted tokens a sequence on medium contexts: latency counts
        dict(name="draft_tokens", op="prompt", shape="mlra4", e4m3=False, batch=4, q_lo=5, q_hi=5, past_lo=700,
             past_hi=1500, lens_seed=1),
        # a packed batch of whole prompts, from one token up, odd lengths
        dict(name="prompts_ragged", op="prompt", shape="mlra4", e4m3=False, batch=24, q_lo=1, q_hi=2047, past_lo=0,
             past_hi=0, lens_seed=2),
        # chunked prefill: the next chunk of two long prompts, over an E4M3 cache
        dict(name="chunk_e4m3", op="prompt", shape="mlra4", e4m3=True, batch=2, q_lo=1000, q_hi=1024, past_lo=6000,
             past_hi=14000, lens_seed=3),
        # one long prompt
        dict(name="prompt_16k", op="prompt", shape="mlra4", e4m3=False, batch=1, q_lo=16384, q_hi=16384, past_lo=0,
             past_hi=0, lens_seed=4),
        # two blocks of 256 (MLRA-2), contexts up to the decode workload's 4096
        dict(name="prompts_mlra2", op="prompt", shape="mlra2", e4m3=False, batch=4, q_lo=1500, q_hi=4096, past_lo=0,
             past_hi=0, lens_seed=5),
        # ---- decode steps over shared prefixes ----
        # a few samples of one short prompt: latency counts
        dict(name="samples_b4", op="shared", shape="mlra4", groups=1, batch=4, pre_lo=1000, pre_hi=1000, suf_lo=0,
             suf_hi=64, lens_seed=6),
        # the headline decode batch and context as one shared prompt with its own continuations
        dict(name="samples_b32_n8192", op="shared", shape="mlra4", groups=1, batch=32, pre_lo=8192, pre_hi=8192,
             suf_lo=1, suf_hi=512, lens_seed=7),
        # several prompts of different lengths (one may be absent), uneven numbers of samples
        dict(name="groups_ragged_mlra2", op="shared", shape="mlra2", groups=6, batch=64, pre_lo=0, pre_hi=12000,
             suf_lo=0, suf_hi=700, lens_seed=8),
        # a long system prompt shared by a large batch
        dict(name="samples_b128_n32768", op="shared", shape="mlra4", groups=1, batch=128, pre_lo=32768,
             pre_hi=32768, suf_lo=64, suf_hi=1024, lens_seed=9),
        # ---- pages of the cache ----
        # a few samples forked from running sequences
        dict(name="fork_8", op="fork", rows=16, len_lo=100, len_hi=2000, slack=64, forks=8, lens_seed=10),
        # a scheduler's turn of a large batch on long contexts
        dict(name="turn_b256", op="turn", rows=256, len_lo=100, len_hi=4096, slack=1000, forks=64, lens_seed=11),
        # compaction of a pool that half its sequences have left
        dict(name="compact_8k", op="compact", rows=128, len_lo=500, len_hi=8000, slack=500, forks=0, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "shared", "shared", "fork", "turn", "compact"])
    seed = rng.randrange(1 << 30)
    if op == "prompt":
        shape = rng.choice(["mlra4", "mlra4", "mlra4", "mlra2", "mla", "rank4"])
        batch = _log_int(rng, 1, 32)
        past = rng.choice([0, _log_int(rng, 1, 16000)])
        q_hi = _log_int(rng, 1, 8000)
        case = dict(op=op, shape=shape, e4m3=shape == "mlra4" and rng.random() < 0.3, batch=batch,
                    q_lo=max(1, int(q_hi * rng.random())), q_hi=q_hi, past_lo=int(past * rng.random()), past_hi=past,
                    lens_seed=seed)
        while _pairs(case) > MAX_PAIRS // 4 or case["batch"] * (case["q_hi"] + case["past_hi"]) > 200000:
            if case["batch"] > 1:
                case["batch"] //= 2
            else:
                case["q_hi"] = max(1, case["q_hi"] // 2)
                case["q_lo"] = min(case["q_lo"], case["q_hi"])
        return case
    if op == "shared":
        groups = rng.choice([1, 1, rng.randint(2, 8)])
        pre = _log_int(rng, 1, 32768)
        suf = _log_int(rng, 1, 1024)
        batch = max(groups, _log_int(rng, 1, 128))
        shape = rng.choice(["mlra4", "mlra4", "mlra2", "mla", "rank4"])
        if shape == "mla":
            batch, groups = min(batch, 64), min(groups, 64)
        return dict(op=op, shape=shape, groups=groups, batch=batch, pre_lo=int(pre * rng.random()), pre_hi=pre,
                    suf_lo=int(suf * rng.random()), suf_hi=suf, lens_seed=seed)
    rows = _log_int(rng, 4, 256)
    hi = _log_int(rng, 20, 8000)
    while rows * hi > 600000:
        hi //= 2
    return dict(op=op, rows=rows, len_lo=int(hi * rng.random()), len_hi=hi, slack=_log_int(rng, 300, 2000),
                forks=0 if op == "compact" else rng.randint(1, max(1, rows // 4)), lens_seed=seed)


# ----------------------------------------------------------------------------------------
# lengths of a case (plain values give the ranges, lens_seed the draw)
# ----------------------------------------------------------------------------------------
def _prompt_lens(case):
    rng = random.Random(case["lens_seed"])
    n = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(case["batch"])]
    return n, past


def _pairs(case):
    n, past = _prompt_lens(case)
    return SHAPES[case["shape"]][1] * sum(q * p + q * (q + 1) // 2 for q, p in zip(n, past))


def _shared_lens(case):
    rng = random.Random(case["lens_seed"])
    cuts = sorted(rng.sample(range(1, case["batch"]), case["groups"] - 1)) if case["groups"] > 1 else []
    offsets = [0] + cuts + [case["batch"]]
    pre = [rng.randint(case["pre_lo"], case["pre_hi"]) for _ in range(case["groups"])]
    suf = [rng.randint(case["suf_lo"], case["suf_hi"]) for _ in range(case["batch"])]
    return offsets, pre, suf


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def _page_plan(case):
    """Rows of a running batch: half or more of them hold sequences, the others are free. Returns
    lens (per row), rows to free, (row, new length) to reserve, (source, destination) to fork,
    the number of pages and the table's width."""
    rng = random.Random(case["lens_seed"])
    rows = case["rows"] + case["forks"]
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["rows"])] + [0] * case["forks"]
    order = list(range(rows))
    rng.shuffle(order)                     # free rows lie among the others
    lens = [lens[i] for i in order]
    live = [i for i in range(rows) if order[i] < case["rows"]]
    empty = [i for i in range(rows) if order[i] >= case["rows"]]
    gone = live[: case["rows"] // 2] if case["op"] == "compact" else (
        rng.sample(live, case["rows"] // 8) if case["op"] == "turn" else [])
    stay = [i for i in live if i not in set(gone)]
    grow = [(i, lens[i] + rng.choice([1, 1, 1, rng.randint(2, 300)])) for i in stay] if case["op"] == "turn" else []
    forks = [(rng.choice(stay), d) for d in empty]
    longest = max([1] + lens + [n for _, n in grow])
    pages = sum(_pages_of(n) for n in lens) + sum(_pages_of(n) - _pages_of(lens[i]) for i, n in grow) + len(forks)
    return lens, gone, grow, forks, pages + case["slack"], _pages_of(longest) + 1


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _paged(g, lens, extra, width, e4m3=False):
    """A pool whose pages are placed by a permutation, and each sequence's row of page ids."""
    used = sum(_pages_of(n) for n in lens)
    num = max(1, used + extra)
    perm = torch.randperm(num, generator=g, device="cuda")[:used].to(torch.int32)
    stride = max([1] + [_pages_of(n) for n in lens])
    table = torch.full((len(lens), stride), -1, dtype=torch.int32, device="cuda")
    off = 0
    for b, n in enumerate(lens):
        table[b, :_pages_of(n)] = perm[off:off + _pages_of(n)]
        off += _pages_of(n)
    pool = torch.empty(num, PAGE, width, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
    for i in range(0, num, 1024):
        part = _randn(g, min(1024, num - i), PAGE, width)
        pool[i:i + 1024] = (part.float() / E4M3_SCALE).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else part
    return pool, table


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _layer(g, shape):
    k, h, d_h, d_c, d_r = SHAPES[shape]
    d_b = d_c // k
    w_uk = (torch.randn(h, d_b, d_h, generator=g, device="cuda") / math.sqrt(d_b)).to(torch.bfloat16)
    w_uv = (torch.randn(h, d_b, d_h, generator=g, device="cuda") / math.sqrt(d_b)).to(torch.bfloat16)
    return w_uk, w_uv


def _handle(shape, w_uk, w_uv, e4m3=False):
    import rank_latent_kv_mlra_b200 as M
    k, h, d_h, d_c, d_r = SHAPES[shape]
    fp8 = dict(cache_fp8=True, latent_scale=E4M3_SCALE, rope_scale=E4M3_SCALE) if e4m3 else {}
    return M.mlra_create(h, d_h, d_c, d_r, k, w_uk, w_uv, **fp8)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "prompt":
        k, h, d_h, d_c, d_r = SHAPES[case["shape"]]
        n, past = _prompt_lens(case)
        w_uk, w_uv = _layer(g, case["shape"])
        total = [a + b for a, b in zip(n, past)]
        pool, table = _paged(g, total, 3, d_c + d_r, case["e4m3"])
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        st = dict(case=case, w_uk=w_uk, w_uv=w_uv, pool=pool, table=table, n=n, total=total, cu_host=cu, cu=_int32(cu),
                  lens=_int32(total), q=_randn(g, cu[-1], h, d_h + d_r),
                  out=torch.empty(cu[-1], h, d_h, dtype=torch.bfloat16, device="cuda"))
        if own:
            import rank_latent_kv_mlra_b200 as M
            st["handle"] = _handle(case["shape"], w_uk, w_uv, case["e4m3"])
            st["ws"] = torch.empty(M.mlra_prefill_workspace_size(st["handle"], cu[-1], len(n), table.shape[1]),
                                   dtype=torch.uint8, device="cuda")
        return st
    if case["op"] == "shared":
        k, h, d_h, d_c, d_r = SHAPES[case["shape"]]
        offsets, pre, suf = _shared_lens(case)
        w_uk, w_uv = _layer(g, case["shape"])
        pool, table = _paged(g, pre + suf, 3, d_c + d_r)
        G, B = case["groups"], case["batch"]
        st = dict(case=case, w_uk=w_uk, w_uv=w_uv, pool=pool, offsets_host=offsets, pre_host=pre, suf_host=suf,
                  pre_table=table[:G].contiguous(), suf_table=table[G:, :max(1, _pages_of(max(suf)))].contiguous(),
                  pre=_int32(pre), suf=_int32(suf), offsets=_int32(offsets), q=_randn(g, B, h, d_h + d_r),
                  out=torch.empty(B, h, d_h, dtype=torch.bfloat16, device="cuda"))
        if own:
            import rank_latent_kv_mlra_b200 as M
            st["handle"] = _handle(case["shape"], w_uk, w_uv)
            st["ws"] = torch.empty(M.mlra_decode_prefix_workspace_size(st["handle"], B, G), dtype=torch.uint8,
                                   device="cuda")
        return st
    lens, gone, grow, forks, pages, stride = _page_plan(case)
    k, h, d_h, d_c, d_r = SHAPES["mlra4"]
    rows = len(lens)
    pool = torch.empty(pages, PAGE, d_c + d_r, dtype=torch.bfloat16, device="cuda")
    for i in range(0, pages, 1024):
        pool[i:i + 1024] = _randn(g, min(1024, pages - i), PAGE, d_c + d_r)
    # page ids of the sequences: a draw of the whole pool, as a pool in use for a while has them
    used = sum(_pages_of(n) for n in lens)
    perm = torch.randperm(pages, generator=g, device="cuda")[:used].to(torch.int32)
    meta = torch.zeros(pages + rows * stride + rows, dtype=torch.int32, device="cuda")
    refs, table, slens = meta[:pages], meta[pages:pages + rows * stride].view(rows, stride), meta[-rows:]
    table.fill_(-1)
    off = 0
    for b, n in enumerate(lens):
        table[b, :_pages_of(n)] = perm[off:off + _pages_of(n)]
        off += _pages_of(n)
    refs[perm.long()] = 1
    slens.copy_(_int32(lens))
    if case["op"] == "compact":            # the sequences that left
        for b in gone:
            refs[table[b, :_pages_of(lens[b])].long()] = 0
            slens[b] = 0
    st = dict(case=case, pool=pool, meta=meta, meta0=meta.clone(), refs=refs, table=table, lens=slens,
              gone=_int32(gone), grow_ids=_int32([i for i, _ in grow]), grow_lens=_int32([n for _, n in grow]),
              src=_int32([s for s, _ in forks]), dst=_int32([d for _, d in forks]))
    if own:
        import rank_latent_kv_mlra_b200 as M
        w_uk, w_uv = _layer(g, "mlra4")
        st["handle"] = _handle("mlra4", w_uk, w_uv)
        st["ws"] = torch.empty(M.mlra_pages_workspace_size(st["handle"], pages, rows), dtype=torch.uint8, device="cuda")
    return st


# ----------------------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------------------
def _rows32(pool, pages, n, e4m3):
    rows = pool[pages[:_pages_of(n)].long()].reshape(-1, pool.shape[2])[:n]
    return rows.view(torch.float8_e4m3fn).float() * E4M3_SCALE if e4m3 else rows.float()


def _plain_prompt(st):
    case = st["case"]
    k, h, d_h, d_c, d_r = SHAPES[case["shape"]]
    d_b, hb, scale = d_c // k, h // k, 1.0 / math.sqrt(d_h + d_r)
    out = torch.empty(st["cu_host"][-1], h, d_h, dtype=torch.bfloat16, device="cuda")
    w_uk, w_uv = st["w_uk"].float(), st["w_uv"].float()
    for b, (n, total) in enumerate(zip(st["n"], st["total"])):
        rows = _rows32(st["pool"], st["table"][b], total, case["e4m3"])
        past, base = total - n, st["cu_host"][b]
        step = max(1, min(n, (1 << 28) // (hb * total)))
        for j in range(k):
            key = torch.cat([rows[:, j * d_b:(j + 1) * d_b], rows[:, d_c:]], dim=1)
            heads = slice(j * hb, (j + 1) * hb)
            for i in range(0, n, step):
                m = min(step, n - i)
                lim = past + i + m                                             # keys any of these queries sees
                q = st["q"][base + i:base + i + m, heads].float().transpose(0, 1)    # [hb][m][d]
                q = torch.cat([q[..., :d_h] @ w_uk[heads].transpose(1, 2), q[..., d_h:]], dim=2) * scale
                s = (q.reshape(hb * m, -1) @ key[:lim].t()).view(hb, m, lim)
                pos = torch.arange(past + i, lim, device="cuda")[:, None]
                s.masked_fill_(torch.arange(lim, device="cuda")[None, :] > pos, float("-inf"))
                s -= s.amax(dim=2, keepdim=True)
                s.exp_()
                z = s.sum(dim=2, keepdim=True)
                o = (s.view(hb * m, lim) @ key[:lim, :d_b]).view(hb, m, d_b) / z
                out[base + i:base + i + m, heads] = (o @ w_uv[heads]).transpose(0, 1).to(torch.bfloat16)
    return out


def _plain_shared(st):
    case = st["case"]
    k, h, d_h, d_c, d_r = SHAPES[case["shape"]]
    d_b, hb, scale = d_c // k, h // k, 1.0 / math.sqrt(d_h + d_r)
    B = case["batch"]
    w_uk, w_uv = st["w_uk"].float(), st["w_uv"].float()
    q = st["q"].float()
    qa = torch.cat([torch.einsum("bhd,hcd->bhc", q[..., :d_h], w_uk), q[..., d_h:]], dim=2) * scale
    lat = torch.zeros(B, h, d_b, device="cuda")
    for grp in range(case["groups"]):
        pre = _rows32(st["pool"], st["pre_table"][grp], st["pre_host"][grp], False)
        b0, b1 = st["offsets_host"][grp], st["offsets_host"][grp + 1]
        for j in range(k):
            heads = slice(j * hb, (j + 1) * hb)
            pkey = torch.cat([pre[:, j * d_b:(j + 1) * d_b], pre[:, d_c:]], dim=1)
            # the prefix, once for all the group's members
            ps = qa[b0:b1, heads].reshape((b1 - b0) * hb, -1) @ pkey.t()
            pm = ps.amax(dim=1, keepdim=True) if ps.shape[1] else torch.full_like(ps[:, :0].sum(1, True), float("-inf"))
            pe = (ps - pm).exp_() if ps.shape[1] else ps
            pz = pe.sum(dim=1, keepdim=True).view(b1 - b0, hb, 1)
            po = (pe @ pkey[:, :d_b]).view(b1 - b0, hb, d_b)
            pm = pm.view(b1 - b0, hb, 1)
            for b in range(b0, b1):
                m, z, o = pm[b - b0], pz[b - b0], po[b - b0]
                if st["suf_host"][b]:
                    suf = _rows32(st["pool"], st["suf_table"][b], st["suf_host"][b], False)
                    key = torch.cat([suf[:, j * d_b:(j + 1) * d_b], suf[:, d_c:]], dim=1)
                    s = qa[b, heads] @ key.t()
                    m2 = torch.maximum(m, s.amax(dim=1, keepdim=True))
                    e, f = (s - m2).exp_(), (m - m2).exp()
                    z = z * f + e.sum(dim=1, keepdim=True)
                    o = o * f + e @ key[:, :d_b]
                if st["suf_host"][b] or st["pre_host"][grp]:
                    lat[b, heads] = o / z
    return torch.einsum("bhc,hcd->bhd", lat, w_uv).to(torch.bfloat16)


def _plain_free(st):
    ids = st["gone"].long()
    stride = st["table"].shape[1]
    held = torch.arange(stride, device="cuda")[None, :] < ((st["lens"][ids] + PAGE - 1) // PAGE)[:, None]
    entry = st["table"][ids].long()
    st["refs"].index_add_(0, torch.where(held, entry, 0).reshape(-1), -held.reshape(-1).to(torch.int32))
    st["lens"][ids] = 0


def _plain_first_free(st, n):
    """Page ids of the first n free pages, in ascending order."""
    rank = torch.cumsum((st["refs"] == 0).to(torch.int32), 0, dtype=torch.int32)
    return torch.searchsorted(rank, torch.arange(1, n + 1, dtype=torch.int32, device="cuda"), out_int32=True)


def _plain_reserve(st):
    ids, stride = st["grow_ids"].long(), st["table"].shape[1]
    old, new = (st["lens"][ids] + PAGE - 1) // PAGE, (st["grow_lens"] + PAGE - 1) // PAGE
    col = torch.arange(stride, device="cuda")[None, :]
    fresh = (col >= old[:, None]) & (col < new[:, None])                        # in (sequence, page) order
    rank = torch.cumsum(fresh.reshape(-1).to(torch.int32), 0, dtype=torch.int32).view(fresh.shape)
    free_rank = torch.cumsum((st["refs"] == 0).to(torch.int32), 0, dtype=torch.int32)
    page = torch.searchsorted(free_rank, rank.contiguous(), out_int32=True)
    st["table"][ids] = torch.where(fresh, page, st["table"][ids])
    st["refs"].index_add_(0, torch.where(fresh, page, 0).reshape(-1).long(), fresh.reshape(-1).to(torch.int32))
    st["lens"][ids] = st["grow_lens"]


def _plain_fork(st):
    src, dst, stride = st["src"].long(), st["dst"].long(), st["table"].shape[1]
    n = st["lens"][src]
    full, part = n // PAGE, n % PAGE
    need = part > 0
    rank = torch.cumsum(need.to(torch.int32), 0, dtype=torch.int32)
    free_rank = torch.cumsum((st["refs"] == 0).to(torch.int32), 0, dtype=torch.int32)
    page = torch.searchsorted(free_rank, rank, out_int32=True)
    col = torch.arange(stride, device="cuda")[None, :]
    entry = st["table"][src]
    shared = col < full[:, None]
    last = need[:, None] & (col == full[:, None])
    st["table"][dst] = torch.where(shared, entry, torch.where(last, page[:, None], st["table"][dst]))
    st["refs"].index_add_(0, torch.where(shared, entry, 0).reshape(-1).long(), shared.reshape(-1).to(torch.int32))
    st["refs"].index_add_(0, torch.where(need, page, 0).long(), need.to(torch.int32))
    st["lens"][dst] = n
    # the rows of each partly filled last page; a fork without one writes its source page's own rows back
    from_page = entry.gather(1, torch.clamp(full, max=stride - 1)[:, None].long())[:, 0].long().clamp(min=0)
    to_page = torch.where(need, page.long(), from_page)
    row = torch.arange(PAGE, device="cuda")[None, :, None]
    st["pool"][to_page] = torch.where(row < part[:, None, None], st["pool"][from_page], st["pool"][to_page])


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    pages = refs.shape[0]
    used = refs > 0
    ids = torch.arange(pages, device="cuda")
    U = used.sum()
    hole, high = ~used & (ids < U), used & (ids >= U)
    # the i-th high page moves to the i-th hole; every other page stays
    hole_rank = torch.cumsum(hole.to(torch.int32), 0, dtype=torch.int32)
    high_rank = torch.cumsum(high.to(torch.int32), 0, dtype=torch.int32)
    moved_to = torch.searchsorted(hole_rank, high_rank, out_int32=True)
    to = torch.where(high, moved_to, ids.to(torch.int32))
    moved_from = torch.searchsorted(high_rank, hole_rank, out_int32=True)
    frm = torch.where(hole, moved_from, ids.to(torch.int32)).long()
    new_refs = torch.where(high, 0, refs[frm])
    st["pool"].copy_(st["pool"][frm])
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    held = col < ((st["lens"] + PAGE - 1) // PAGE)[:, None]
    table.copy_(torch.where(held, to[table.long().clamp(min=0)], table))
    refs.copy_(new_refs)


# ----------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------
def run(state):
    st = state
    op = st["case"]["op"]
    if own:
        import rank_latent_kv_mlra_b200 as M
    if op == "prompt":
        if not own:
            return _plain_prompt(st)
        M.mlra_prefill(st["handle"], st["q"], st["cu"], st["pool"], st["table"], st["lens"], st["out"],
                       workspace=st["ws"])
        return st["out"]
    if op == "shared":
        if not own:
            return _plain_shared(st)
        M.mlra_decode_prefix(st["handle"], st["q"], st["pool"], st["pre_table"], st["pre"], st["offsets"],
                             st["suf_table"], st["suf"], st["out"], workspace=st["ws"])
        return st["out"]
    st["meta"].copy_(st["meta0"])          # the turn's page counts, tables and lengths
    if not own:
        if op == "turn":
            _plain_free(st)
            _plain_reserve(st)
        if op in ("turn", "fork"):
            _plain_fork(st)
        if op == "compact":
            _plain_compact(st)
    else:
        pages = (st["refs"], st["table"], st["lens"])
        if op == "turn":
            M.mlra_free_pages(st["handle"], *pages, st["gone"], workspace=st["ws"])
            M.mlra_reserve_pages(st["handle"], *pages, st["grow_ids"], st["grow_lens"], workspace=st["ws"])
        if op in ("turn", "fork"):
            M.mlra_fork_pages(st["handle"], st["pool"], *pages, st["src"], st["dst"], workspace=st["ws"])
        if op == "compact":
            M.mlra_compact_pages(st["handle"], st["pool"], *pages, workspace=st["ws"])
    return {"refs": st["refs"], "table": st["table"], "lens": st["lens"], "pool": st["pool"]}


# ----------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "prompt":
        k, h, d_h, d_c, d_r = SHAPES[case["shape"]]
        n, past = _prompt_lens(case)
        d_b, T = d_c // k, sum(n)
        rows = sum(a + b for a, b in zip(n, past))
        pairs = _pairs(case)
        # over the latent (absorbed query, up-projected result) or over each head's own keys and values
        latent = pairs * 2 * (2 * d_b + d_r) + T * h * 4 * d_b * d_h
        per_head = pairs * 2 * (2 * d_h + d_r) + rows * h * 4 * d_b * d_h
        size = 1 if case["e4m3"] else 2
        nbytes = rows * (d_c + d_r) * size + T * h * (2 * d_h + d_r) * 2 + 2 * h * d_b * d_h * 2
        return {"bytes": nbytes, "flops": min(latent, per_head)}
    if case["op"] == "shared":
        k, h, d_h, d_c, d_r = SHAPES[case["shape"]]
        offsets, pre, suf = _shared_lens(case)
        d_b, B = d_c // k, case["batch"]
        pairs = h * (sum(p * (b - a) for p, a, b in zip(pre, offsets, offsets[1:])) + sum(suf))
        nbytes = (sum(pre) + sum(suf)) * (d_c + d_r) * 2 + B * h * (2 * d_h + d_r) * 2 + 2 * h * d_b * d_h * 2
        return {"bytes": nbytes, "flops": pairs * 2 * (2 * d_b + d_r) + B * h * 4 * d_b * d_h}
    lens, gone, grow, forks, pages, stride = _page_plan(case)
    k, h, d_h, d_c, d_r = SHAPES["mlra4"]
    row_bytes = (d_c + d_r) * 2
    nbytes = 4 * pages                                                     # the counts are looked through
    if case["op"] in ("turn", "fork"):
        nlen = dict(grow)
        nbytes += sum(2 * row_bytes * (nlen.get(s, lens[s]) % PAGE) + 16 * _pages_of(lens[s]) for s, _ in forks)
        nbytes += sum(12 * _pages_of(lens[i]) for i in gone) + 16 * len(grow)
    if case["op"] == "compact":
        used = sum(_pages_of(n) for i, n in enumerate(lens) if i not in set(gone))
        # used pages are spread over the whole pool: this share of them lies past the first `used`
        moved = int(used * (1 - used / pages))
        nbytes += moved * 2 * PAGE * row_bytes + 8 * used
    return {"bytes": nbytes, "flops": 0}


# ----------------------------------------------------------------------------------------
# 64-bit results, from the definitions
# ----------------------------------------------------------------------------------------
def _rows64(pool, pages, n, e4m3):
    ids = pages[:_pages_of(n)].to(torch.int64)
    rows = torch.index_select(pool, 0, ids).flatten(0, 1)[:n]
    if e4m3:
        return rows.view(torch.float8_e4m3fn).to(torch.float64) * E4M3_SCALE
    return rows.to(torch.float64)


def _attend64(q, rows, w_uk, w_uv, shape, first_pos):
    """Heads' outputs for queries q [m][h][.] at positions first_pos, first_pos + 1, ... (None:
    every query sees every row), with each head's own keys and values."""
    k, h, d_h, d_c, d_r = SHAPES[shape]
    d_b, hb = d_c // k, h // k
    m, n = q.shape[0], rows.shape[0]
    out = torch.zeros(m, h, d_h, dtype=torch.float64, device="cuda")
    if n == 0:
        return out
    kr = rows[:, d_c:]
    for head in range(h):
        block = rows[:, (head // hb) * d_b:(head // hb + 1) * d_b]
        key = torch.cat([block @ w_uk[head], kr], dim=1)
        val = block @ w_uv[head]
        step = max(1, (1 << 27) // n)
        for i in range(0, m, step):
            qi = q[i:i + step, head]
            seen = n if first_pos is None else min(n, first_pos + i + qi.shape[0])
            s = torch.mm(qi, key[:seen].t()) / math.sqrt(d_h + d_r)
            if first_pos is not None:
                s = s + torch.triu(torch.full_like(s, float("-inf")), diagonal=first_pos + i + 1)
            out[i:i + step, head] = torch.softmax(s, dim=1) @ val[:seen]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prompt":
        w_uk, w_uv = st["w_uk"].to(torch.float64), st["w_uv"].to(torch.float64)
        parts = []
        for b, (n, total) in enumerate(zip(st["n"], st["total"])):
            rows = _rows64(st["pool"], st["table"][b], total, case["e4m3"])
            q = st["q"][st["cu_host"][b]:st["cu_host"][b + 1]].to(torch.float64)
            parts.append(_attend64(q, rows, w_uk, w_uv, case["shape"], total - n))
        return torch.cat(parts)
    if case["op"] == "shared":
        w_uk, w_uv = st["w_uk"].to(torch.float64), st["w_uv"].to(torch.float64)
        offsets, parts = st["offsets_host"], []
        if case["batch"] * SHAPES[case["shape"]][1] * (max(st["pre_host"]) + 1024) > 1 << 29:
            return _exact_shared_blocked(st)
        for grp in range(case["groups"]):
            pre = _rows64(st["pool"], st["pre_table"][grp], st["pre_host"][grp], False)
            for b in range(offsets[grp], offsets[grp + 1]):
                suf = _rows64(st["pool"], st["suf_table"][b], st["suf_host"][b], False)
                parts.append(_attend64(st["q"][b:b + 1].to(torch.float64), torch.cat([pre, suf]), w_uk, w_uv,
                                       case["shape"], None))
        return torch.cat(parts)
    return _exact_pages(st)


def _exact_shared_blocked(st):
    """The same for large batches: each head's keys and values of a prefix are formed once."""
    case = st["case"]
    k, h, d_h, d_c, d_r = SHAPES[case["shape"]]
    d_b, hb = d_c // k, h // k
    w_uk, w_uv = st["w_uk"].to(torch.float64), st["w_uv"].to(torch.float64)
    out = torch.zeros(case["batch"], h, d_h, dtype=torch.float64, device="cuda")
    for grp in range(case["groups"]):
        b0, b1 = st["offsets_host"][grp], st["offsets_host"][grp + 1]
        pre = _rows64(st["pool"], st["pre_table"][grp], st["pre_host"][grp], False)
        sufs = [_rows64(st["pool"], st["suf_table"][b], st["suf_host"][b], False) for b in range(b0, b1)]
        own_rows = torch.cat([pre] + sufs)
        owner = torch.tensor([-1] * len(pre) + [i for i, s in enumerate(sufs) for _ in range(len(s))], device="cuda")
        mask = (owner[None, :] != -1) & (owner[None, :] != torch.arange(b1 - b0, device="cuda")[:, None])
        if own_rows.shape[0] == 0:
            continue
        for head in range(h):
            block = own_rows[:, (head // hb) * d_b:(head // hb + 1) * d_b]
            key = torch.cat([block @ w_uk[head], own_rows[:, d_c:]], dim=1)
            s = st["q"][b0:b1, head].to(torch.float64) @ key.t() / math.sqrt(d_h + d_r)
            p = torch.softmax(s.masked_fill(mask, float("-inf")), dim=1)
            out[b0:b1, head] = torch.nan_to_num(p) @ (block @ w_uv[head])
    return out


def _exact_pages(st):
    """The page operators one page at a time, on the host."""
    op = st["case"]["op"]
    refs, table, lens = (st[x].cpu().numpy().astype(np.int64) for x in ("refs", "table", "lens"))
    pool = st["pool"].clone()
    free = [i for i in range(len(refs)) if refs[i] == 0]
    if op == "turn":
        for b in st["gone"].tolist():
            for p in table[b, :_pages_of(int(lens[b]))]:
                refs[p] -= 1
            lens[b] = 0
        free = [i for i in range(len(refs)) if refs[i] == 0]
        for b, n in zip(st["grow_ids"].tolist(), st["grow_lens"].tolist()):
            for c in range(_pages_of(int(lens[b])), _pages_of(n)):
                table[b, c] = free.pop(0)
                refs[table[b, c]] = 1
            lens[b] = n
    if op in ("turn", "fork"):
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            n = int(lens[s])
            for c in range(n // PAGE):
                table[d, c] = table[s, c]
                refs[table[s, c]] += 1
            if n % PAGE:
                page = free.pop(0)
                table[d, n // PAGE] = page
                refs[page] = 1
                pool[page, :n % PAGE] = st["pool"][int(table[s, n // PAGE]), :n % PAGE]
            lens[d] = n
    if op == "compact":
        count = int((refs > 0).sum())
        holes = [i for i in range(count) if refs[i] == 0]
        high = [i for i in range(count, len(refs)) if refs[i] > 0]
        place = dict(zip(high, holes))
        for a, b in place.items():
            refs[b], refs[a] = refs[a], 0
        if high:
            pool[torch.tensor(holes, device="cuda")] = st["pool"][torch.tensor(high, device="cuda")]
        for b in range(len(lens)):
            for c in range(_pages_of(int(lens[b]))):
                table[b, c] = place.get(int(table[b, c]), table[b, c])
    return {"refs": torch.from_numpy(refs), "table": torch.from_numpy(table), "lens": torch.from_numpy(lens),
            "pool": pool.to(torch.float64)}
