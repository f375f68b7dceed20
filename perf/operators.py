"""Cases, inputs and plain forms of the operators that work on the whole paged cache:
attention of new tokens over it, attention over blocks of it that a cheap score selects,
the block keys and scores behind that selection, and reading cached rows back.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, calls
this repository's library for it on the same state.  ``exact`` computes the same in 64 bits.
"""
import math

import torch

own = False

PAGE = 64
LATENT, ROPE, BLOCK = 512, 64, 128          # latent dims, RoPE dims, dims under one scale
IDX_HEADS, IDX_DIM = 64, 128                # indexer heads and their dims
IDX_PAGE = PAGE * (IDX_DIM + 4)             # indexer page: 64 keys, then 64 fp32 scales
ROW = {"ds": 656, "e4m3": 576, "bf16": 1152}   # latent row bytes of the three pool formats
PLAIN_SCALE = 8.0 / 448.0                   # pool scale of a plain e4m3 pool
SSMAX = 0.4
SIGMA = 576 ** -0.5
E4M3 = torch.float8_e4m3fn


# ---- cases ------------------------------------------------------------------------

def listed():
    return [
        # one request's new token, one GPU's 16 heads, a short context: latency counts
        dict(name="paged_tiny", op="paged", requests=1, q=1, lo=4096, hi=4096, heads=16, rope=64, fmt="ds",
             ssmax=False, window=0),
        # a decode batch of uneven contexts, 16 heads: bound by the cache's bytes
        dict(name="paged_batched", op="paged", requests=32, q=1, lo=8192, hi=65536, heads=16, rope=64, fmt="ds",
             ssmax=False, window=0),
        # a speculative verification step, all 128 heads: bound by the matrix products
        dict(name="paged_spec", op="paged", requests=8, q=4, lo=60000, hi=60000, heads=128, rope=64, fmt="ds",
             ssmax=True, window=0),
        # a draft layer: the last 2,048 tokens of each request, an unquantised cache, odd lengths from 1 up
        dict(name="paged_window", op="paged", requests=63, q=1, lo=1, hi=20011, heads=16, rope=64, fmt="bf16",
             ssmax=False, window=2048),
        # one request of a million tokens, a layer without RoPE, one scale for the whole pool
        dict(name="paged_long", op="paged", requests=1, q=1, lo=1048576, hi=1048576, heads=32, rope=0, fmt="e4m3",
             ssmax=False, window=0),
        # the decode batch again, 32 selected blocks (2,048 tokens) of each context
        dict(name="block_batched", op="block", requests=32, q=1, lo=8192, hi=65536, heads=16, rope=64, fmt="ds",
             ssmax=False, blocks=32),
        # the verification step over selected blocks
        dict(name="block_spec", op="block", requests=8, q=4, lo=60000, hi=60000, heads=128, rope=64, fmt="ds",
             ssmax=True, blocks=32),
        # a million tokens, an odd number of blocks, odd length
        dict(name="block_long", op="block", requests=1, q=4, lo=1048001, hi=1048001, heads=128, rope=0, fmt="e4m3",
             ssmax=False, blocks=45),
        # a decode step: the few pages that just filled, then every request's block scores
        dict(name="index_decode", op="index", requests=32, q=1, lo=8192, hi=65536, ssmax=False, fresh=1),
        # a prompt's last chunk: every page's key, then the scores of 2,048 queries
        dict(name="index_prefill", op="index", requests=1, q=2048, lo=32768, hi=32768, ssmax=True, fresh=512),
        # a cached prefix read back for the next chunk of its prompt
        dict(name="read_prefix", op="read", rows=30720, pool=512, fmt="ds", rope=64, skip=0),
        # a few scattered rows of one-scale cache, some of them padding
        dict(name="read_ragged", op="read", rows=701, pool=97, fmt="e4m3", rope=64, skip=13),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["paged", "paged", "paged", "block", "block", "index", "read"])
    if op == "read":
        pool = _between(rng, 1, 600)
        rows = _between(rng, 1, pool * PAGE)
        return dict(op=op, rows=rows, pool=pool, fmt=rng.choice(["ds", "e4m3", "bf16"]), rope=rng.choice([64, 64, 0]),
                    skip=rng.choice([0, 0, 5, 17]))
    q = rng.choice([1, 1, 1, 2, 3, 4])
    hi = _between(rng, q, 200000)
    if op == "index":
        q = rng.choice([1, 1, 2, 4, _between(rng, 5, 1024)])
        hi = max(hi, q)
        requests = min(_between(rng, 1, 64), max(1, 1200000 // hi), max(1, 4096 // q))
        lo = _between(rng, q, hi)
        pages = sum(-(-n // PAGE) for n in _lengths(dict(requests=requests, lo=lo, hi=hi, q=q)))
        return dict(op=op, requests=requests, q=q, lo=lo, hi=hi, ssmax=rng.random() < 0.3,
                    fresh=_between(rng, 1, pages))
    heads = rng.choice([16, 16, 32, 64, 128])
    # no more tokens, and no more (token, head) pairs, than the largest listed cases
    most = min(1000000, 240000000 // (q * heads))
    hi = min(hi, most)
    requests = min(_between(rng, 1, 64), max(1, most // hi))
    c = dict(op=op, requests=requests, q=q, lo=_between(rng, q, hi), hi=hi, heads=heads,
             rope=rng.choice([64, 64, 64, 0]), fmt=rng.choice(["ds", "ds", "e4m3", "bf16"]), ssmax=rng.random() < 0.3)
    if op == "block":
        c["blocks"] = _between(rng, 1, 64)
    else:
        c["window"] = rng.choice([0, 0, 0, _between(rng, 1, 8192)])
    return c


def _lengths(case):
    """Every request's cached tokens (its new ones among them): uneven, the same for every seed."""
    lo, hi = case["lo"], case["hi"]
    return [hi if case["requests"] == 1 else lo + int((hi - lo) * ((i + 1) * 0.6180339887498949 % 1.0) + 0.5)
            for i in range(case["requests"])]


def _visible(case):
    """(request, visible length) of every new token, in order."""
    return [(r, n - case["q"] + j + 1) for r, n in enumerate(_lengths(case)) for j in range(case["q"])]


def work(case):
    op = case["op"]
    if op == "read":
        n = case["rows"] - (len(range(0, case["rows"], case["skip"])) if case["skip"] else 0)
        held = {"ds": 528, "e4m3": 512, "bf16": 1024}[case["fmt"]]
        held += {"ds": 128, "e4m3": 64, "bf16": 128}[case["fmt"]] if case["rope"] else 0
        return {"bytes": case["rows"] * 4 + n * (held + 2 * (LATENT + case["rope"]) + 132 + 2 * IDX_DIM), "flops": 0}
    lens, vis, tokens = _lengths(case), _visible(case), case["requests"] * case["q"]
    if op == "index":
        pairs = sum((n - 1) // PAGE for _, n in vis)
        seen = sum((n - 1) // PAGE for n in lens)
        return {"bytes": case["fresh"] * (IDX_PAGE + 4 + 132) + seen * (132 + 4) + pairs * 4 +
                tokens * (IDX_HEADS * IDX_DIM + 4 + 4 * IDX_HEADS),
                "flops": pairs * 2 * IDX_HEADS * IDX_DIM + case["fresh"] * PAGE * IDX_DIM}
    row = {"ds": 528, "e4m3": 512, "bf16": 1024}[case["fmt"]]
    row += {"ds": 128, "e4m3": 64, "bf16": 128}[case["fmt"]] if case["rope"] else 0
    heads, dims = case["heads"], LATENT + case["rope"]
    more = tokens * heads * (2 * dims + 2 * LATENT + 4)     # queries, outputs, log-sum-exps
    if op == "paged":
        w = case["window"]
        pairs = sum(min(n, w) if w else n for _, n in vis)
        rows = sum(min(n, w + case["q"] - 1) if w else n for n in lens)
        return {"bytes": rows * row + rows // PAGE * 4 + more, "flops": 2 * heads * (dims + LATENT) * pairs}
    k = case["blocks"]
    pairs = rows = scores = 0
    for r, n in vis:
        pairs += min(n, (k - 1) * PAGE + (n - 1) % PAGE + 1)
        scores += (n - 1) // PAGE
    for n in lens:                                          # blocks that any of a request's tokens selects
        rows += n * (1 - (1 - min(1.0, k * PAGE / n)) ** case["q"])
    return {"bytes": rows * row + scores * 4 + tokens * (k + 1) * 4 + more, "flops": 2 * heads * (dims + LATENT) * pairs}


# ---- inputs -----------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _quant(x, block):
    """fp32 [n, d] -> e4m3 codes (uint8) and a scale for each `block` values."""
    xb = x.view(x.shape[0], -1, block)
    s = xb.abs().amax(-1) / 448
    return (xb / s[..., None]).to(E4M3).view(torch.uint8).view(x.shape), s


def _latent_pool(g, fmt, rows):
    if fmt == "ds":
        codes, s = _quant(_randn(g, rows, LATENT), BLOCK)
        pe = _randn(g, rows, ROPE).bfloat16()
        return torch.cat([codes, s.view(torch.uint8), pe.view(torch.uint8)], 1)
    x = _randn(g, rows, LATENT + ROPE)
    return (x / PLAIN_SCALE).clamp(-448, 448).to(E4M3).view(torch.uint8) if fmt == "e4m3" else x.bfloat16().view(torch.uint8)


def _index_pool(g, pages):
    codes, s = _quant(_randn(g, pages * PAGE, IDX_DIM), IDX_DIM)
    return torch.cat([codes.view(pages, -1), s.view(pages, PAGE).view(torch.uint8)], 1)


def _layout(case, g):
    """Batch arrays: a shuffled pool, two pages of it nobody's."""
    lens = _lengths(case)
    pages = [-(-n // PAGE) for n in lens]
    order = torch.randperm(sum(pages) + 2, generator=g, device="cuda").int()
    table = torch.zeros(len(lens), max(pages), dtype=torch.int32, device="cuda")
    at = 0
    tails = []
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        tails += [(at + n - 1, i) for i in range((lens[r] - 1) % PAGE + 1, PAGE)]
        at += n
    where = torch.tensor(tails, dtype=torch.long, device="cuda").reshape(-1, 2)
    unused = order[where[:, 0]].long() * PAGE + where[:, 1]       # rows behind the last token of each request
    return dict(case=case, pages=int(sum(pages)) + 2, table=table, order=order[:at], unused=unused, max_ctx=max(lens),
                tokens=len(lens) * case["q"], ctx_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                cu_q=torch.arange(len(lens) + 1, dtype=torch.int32, device="cuda") * case["q"])


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "read":
        n = case["rows"]
        slot = torch.randperm(case["pool"] * PAGE, generator=g, device="cuda")[:n].int()
        if case["skip"]:
            slot[::case["skip"]] = -1
        return dict(case=case, slot=slot, latent=_latent_pool(g, case["fmt"], case["pool"] * PAGE),
                    index=_index_pool(g, case["pool"]),
                    c=torch.zeros(n, LATENT, dtype=torch.bfloat16, device="cuda"),
                    k_pe=torch.zeros(n, ROPE, dtype=torch.bfloat16, device="cuda") if case["rope"] else None,
                    k=torch.zeros(n, IDX_DIM, dtype=torch.bfloat16, device="cuda"))
    s = _layout(case, g)
    t = s["tokens"]
    if case["op"] == "index":
        s["index"] = _index_pool(g, s["pages"])
        codes, scale = _quant(_randn(g, t, IDX_HEADS * IDX_DIM), IDX_HEADS * IDX_DIM)
        s |= dict(iq8=codes.view(t, IDX_HEADS, IDX_DIM), iq_scale=scale.view(t), iw=_randn(g, t, IDX_HEADS) / 8)
        s["block_pool"] = torch.zeros(-(-s["pages"] // PAGE), IDX_PAGE, dtype=torch.uint8, device="cuda")
        _write_block_keys(s, s["order"])                                          # pages of earlier steps
        pick = torch.randperm(len(s["order"]), generator=g, device="cuda")[:case["fresh"]]
        s["fresh"] = s["order"][pick].contiguous()                                # pages that filled just now
        s["index"].view(-1)[(s["fresh"].long() * IDX_PAGE)[:, None] + torch.arange(128, device="cuda")] ^= 0x80
        s["scores"] = torch.zeros(t, s["table"].shape[1], device="cuda")
        return s
    pool = _latent_pool(g, case["fmt"], s["pages"] * PAGE)
    junk = torch.randint(0, 256, (len(s["unused"]), pool.shape[1]), generator=g, device="cuda").byte()
    pool[s["unused"]] = junk                                                      # nobody's rows hold anything
    s |= dict(latent=pool, q=_randn(g, t, case["heads"], LATENT + case["rope"]).bfloat16(),
              out=torch.zeros(t, case["heads"], LATENT, dtype=torch.bfloat16, device="cuda"),
              lse=torch.zeros(t, case["heads"], device="cuda"))
    if case["op"] == "block":
        s["scores"] = _randn(g, t, s["table"].shape[1])
        s["blocks"] = torch.zeros(t, case["blocks"], dtype=torch.int32, device="cuda")
        s["blocks_len"] = torch.zeros(t, dtype=torch.int32, device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------------

def _rows(pool, fmt, rope, at):
    """fp32 latents [..., 512] and RoPE keys [..., 64] (or None) of the pool rows `at`."""
    raw = pool[at]
    if fmt == "ds":
        s = raw[..., 512:528].contiguous().view(torch.float32)
        c = (raw[..., :512].contiguous().view(E4M3).float().view(*at.shape, 4, BLOCK) * s[..., None]).view(*at.shape, LATENT)
        return c, raw[..., 528:].contiguous().view(torch.bfloat16).float() if rope else None
    x = raw.view(E4M3).float() * torch.tensor(PLAIN_SCALE, dtype=torch.float32) if fmt == "e4m3" else raw.view(torch.bfloat16).float()
    return x[..., :LATENT], x[..., LATENT:] if rope else None


def _tokens(s):
    """Request and visible length of every new token."""
    q = s["case"]["q"]
    t = torch.arange(s["tokens"], device="cuda")
    return t // q, s["ctx_len"][t // q].long() - q + t % q + 1


def _attend(s, q, c, k_pe, seen, n):
    """q [G, M, D] over rows [G, L, ...]; seen [G, M, L]; n [G, M]: out [G, M, 512] and lse [G, M], fp32."""
    scale = SIGMA * (SSMAX * torch.log(n.float()) if s["case"]["ssmax"] else torch.ones_like(n, dtype=torch.float32))
    z = q[..., :LATENT] @ c.transpose(1, 2)
    if k_pe is not None:
        z = z + q[..., LATENT:] @ k_pe.transpose(1, 2)
    z = torch.where(seen, z * scale[..., None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    return (p @ c) / l, (m + torch.log(l)).squeeze(-1)


def _paged(s):
    case = s["case"]
    b, rows = case["requests"], case["q"] * case["heads"]
    at = (s["table"].long()[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")).view(b, -1)
    c, k_pe = _rows(s["latent"], case["fmt"], case["rope"], at)
    pos = torch.arange(at.shape[1], device="cuda")
    held = (pos < s["ctx_len"][:, None])[..., None]
    c = torch.where(held, c, 0.0)
    k_pe = torch.where(held, k_pe, 0.0) if k_pe is not None else None
    n = _tokens(s)[1].view(b, case["q"])
    seen = pos < n[..., None]
    if case["window"]:
        seen &= pos >= n[..., None] - case["window"]
    out, lse = _attend(s, s["q"].float().view(b, rows, -1), c, k_pe,
                       seen.repeat_interleave(case["heads"], 1), n.repeat_interleave(case["heads"], 1))
    return dict(out=out.bfloat16().view(s["out"].shape), lse=lse.view(s["lse"].shape))


def _block(s):
    case, k = s["case"], s["case"]["blocks"]
    r, n = _tokens(s)
    full = (n - 1) // PAGE                                       # blocks before the one of the newest token
    col = torch.arange(s["scores"].shape[1], device="cuda")
    order = torch.sort(torch.where(col < full[:, None], s["scores"], -math.inf), dim=-1, descending=True, stable=True).indices
    take = full.clamp(max=k - 1)
    pos = torch.arange(k, device="cuda")
    order = torch.nn.functional.pad(order, (0, max(0, k - order.shape[1])))[:, :k]
    chosen = torch.where(pos < take[:, None], order, 1 << 40).sort(-1).values
    chosen = torch.where(pos == take[:, None], full[:, None], chosen)
    blocks = torch.where(pos <= take[:, None], chosen, -1)
    page = s["table"].long()[r[:, None], blocks.clamp(min=0)]
    inner = torch.arange(PAGE, device="cuda")
    at = (page[..., None] * PAGE + inner).flatten(1)
    where = (blocks[..., None] * PAGE + inner).flatten(1)
    seen = (where >= 0) & (where < n[:, None])
    c, k_pe = _rows(s["latent"], case["fmt"], case["rope"], at)
    c = torch.where(seen[..., None], c, 0.0)
    k_pe = torch.where(seen[..., None], k_pe, 0.0) if k_pe is not None else None
    out, lse = _attend(s, s["q"].float(), c, k_pe, seen[:, None].expand(-1, case["heads"], -1), n[:, None].expand(-1, case["heads"]))
    return dict(blocks=blocks.int(), blocks_len=(take + 1).int(), out=out.bfloat16(), lse=lse)


def _write_block_keys(s, pages):
    """Mean of each page's keys, summed in 64 bits, as e4m3 codes and a scale, into the row of the page's number."""
    p = pages.long()
    raw = s["index"][p]
    keys = raw[:, :PAGE * IDX_DIM].contiguous().view(E4M3).double().view(-1, PAGE, IDX_DIM)
    mean = ((keys * raw[:, PAGE * IDX_DIM:].contiguous().view(torch.float32).double()[..., None]).sum(1) / PAGE).float()
    top = mean.abs().amax(-1)
    scale = torch.where(top > 0, top / 448, 1.0)
    codes = (mean / scale[:, None]).to(E4M3).view(torch.uint8)
    flat = s["block_pool"].view(-1)
    base, row = p // PAGE * IDX_PAGE, p % PAGE
    flat[(base + row * IDX_DIM)[:, None] + torch.arange(IDX_DIM, device="cuda")] = codes
    flat[(base + PAGE * IDX_DIM + row * 4)[:, None] + torch.arange(4, device="cuda")] = scale[:, None].view(torch.uint8)


def _block_pool(s):
    """The block keys' codes and scales, as the values they are."""
    return dict(codes=s["block_pool"][:, :PAGE * IDX_DIM].view(E4M3), scales=s["block_pool"][:, PAGE * IDX_DIM:].view(torch.float32))


def _index(s):
    _write_block_keys(s, s["fresh"])
    case, got = s["case"], _block_pool(s)
    b, t = case["requests"], s["tokens"]
    p = s["table"].long()
    keys = got["codes"].float().view(-1, IDX_DIM)[p.view(-1)].view(b, -1, IDX_DIM)
    scales = got["scales"].contiguous().view(-1)[p.view(-1)].view(b, 1, -1)
    dots = (s["iq8"].view(E4M3).float().view(b, -1, IDX_DIM) @ keys.transpose(1, 2)).relu()
    sums = (dots.view(b, case["q"], IDX_HEADS, -1) * s["iw"].view(b, case["q"], IDX_HEADS, 1)).sum(2)
    n = _tokens(s)[1]
    factor = s["iq_scale"] * (SSMAX * torch.log(n.float()) if case["ssmax"] else 1.0)
    scores = (sums * scales).view(t, -1) * factor[:, None]
    scores = torch.where(torch.arange(p.shape[1], device="cuda") < ((n - 1) // PAGE)[:, None], scores, s["scores"])
    return dict(**got, scores=scores)


def _read(s):
    case, slot = s["case"], s["slot"].long()
    there = slot >= 0
    at = slot.clamp(min=0)
    c, k_pe = _rows(s["latent"], case["fmt"], case["rope"], at)
    page = s["index"][at // PAGE]
    row = at % PAGE
    codes = page.gather(1, (row * IDX_DIM)[:, None] + torch.arange(IDX_DIM, device="cuda")).view(E4M3).float()
    k = codes * page[:, PAGE * IDX_DIM:].view(torch.float32).gather(1, row[:, None])
    keep = lambda new, old: torch.where(there[:, None], new.bfloat16(), old)  # noqa: E731
    return dict(c=keep(c, s["c"]), k_pe=keep(k_pe, s["k_pe"]) if case["rope"] else None, k=keep(k, s["k"]))


# ---- the library's calls ----------------------------------------------------------

def _library(s):
    """What a user's program keeps between calls: the problem, the cache descriptors' pools and a workspace."""
    from sparse_mla_attention_indexer_b200 import sml
    case = s["case"]
    kept = dict(sml=sml)
    if "latent" in s:
        flat = s["latent"].view(-1)
        kept["latent"] = {"ds": flat, "e4m3": sml.E4M3Latent(flat, PLAIN_SCALE), "bf16": sml.Bf16Latent(flat)}[case["fmt"]]
    if case["op"] == "read":
        return kept
    p = sml.make_problem(num_heads=case.get("heads", 16), topk=2048, rope_dim=case.get("rope", 64), cu_q=s["cu_q"],
                         ctx_len=s["ctx_len"], block_table=s["table"], max_ctx=s["max_ctx"], ssmax=case["ssmax"],
                         sm_scale=SIGMA, ssmax_s=SSMAX, ssmax_s_index=SSMAX, num_tokens=s["tokens"])
    kept["ws"] = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(kept["ws"])
    kept["p"] = p
    return kept


def _own(s):
    if "kept" not in s:
        s["kept"] = _library(s)
    kept, op = s["kept"], s["case"]["op"]
    sml = kept["sml"]
    if op == "read":
        sml.sml_latent_cache_read(s["slot"], kept["latent"], s["c"], s["k_pe"])
        sml.sml_indexer_k_cache_read(s["slot"], s["index"], s["k"])
        return dict(c=s["c"], k_pe=s["k_pe"], k=s["k"])
    p, ws = kept["p"], kept["ws"]
    if op == "paged":
        sml.sml_paged_mla_decode(p, s["q"], kept["latent"], s["out"], s["lse"], ws, window=s["case"]["window"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "block":
        sml.sml_block_topk(p, s["scores"], s["blocks"], s["blocks_len"], ws)
        sml.sml_block_mla_decode(p, s["q"], kept["latent"], s["blocks"], s["blocks_len"], s["out"], s["lse"], ws)
        return dict(blocks=s["blocks"], blocks_len=s["blocks_len"], out=s["out"], lse=s["lse"])
    sml.sml_block_keys_write(s["index"], s["fresh"], s["block_pool"], ws)
    sml.sml_block_scores(p, s["iq8"], s["iq_scale"], s["iw"], s["block_pool"], s["scores"], ws)
    return dict(**_block_pool(s), scores=s["scores"])


def run(state):
    if own:
        return _own(state)
    return {"paged": _paged, "block": _block, "index": _index, "read": _read}[state["case"]["op"]](state)


# ---- the definitions in 64 bits ---------------------------------------------------

def _exact_rows(s, rows):
    """Latents and RoPE keys of pool rows, from the byte layouts, in 64 bits."""
    raw = s["latent"].index_select(0, rows)
    fmt = s["case"]["fmt"]
    if fmt == "bf16":
        x = raw.view(torch.bfloat16).double()
        return x[:, :512], x[:, 512:]
    if fmt == "e4m3":
        x = raw.view(E4M3).double() * float(torch.tensor(PLAIN_SCALE, dtype=torch.float32))
        return x[:, :512], x[:, 512:]
    c = torch.cat([raw[:, 128 * b:128 * b + 128].contiguous().view(E4M3).double() *
                   raw[:, 512 + 4 * b:516 + 4 * b].contiguous().view(torch.float32).double() for b in range(4)], 1)
    return c, raw[:, 528:].contiguous().view(torch.bfloat16).double()


def _exact_token(s, t, rows, n):
    """Softmax attention of new token t over pool rows, n visible: out [H, 512], lse [H]."""
    q = s["q"][t].double()
    c, k_pe = _exact_rows(s, rows)
    factor = 576.0 ** -0.5 * (0.4 * math.log(n) if s["case"]["ssmax"] else 1.0)
    z = (q @ torch.cat([c, k_pe], 1).T if s["case"]["rope"] else q @ c.T) * factor
    lse = torch.logsumexp(z, 1)
    return torch.exp(z - lse[:, None]) @ c, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "read":
        got = {"c": s["c"].double(), "k_pe": s["k_pe"].double() if case["rope"] else None, "k": s["k"].double()}
        at = (s["slot"] >= 0).nonzero()[:, 0]
        slot = s["slot"][at].long()
        c, k_pe = _exact_rows(s, slot)
        got["c"][at] = c
        if case["rope"]:
            got["k_pe"][at] = k_pe
        keys = s["index"][:, :8192].contiguous().view(-1, 128).index_select(0, slot).view(E4M3).double()
        got["k"][at] = keys * s["index"][:, 8192:].contiguous().view(torch.float32).view(-1)[slot].double()[:, None]
        return got
    if case["op"] == "index":
        scores = s["scores"].double()
        keys = s["index"][:, :8192].contiguous().view(E4M3).double().view(-1, 64, 128)
        means = torch.einsum("psd,ps->pd", keys, s["index"][:, 8192:].contiguous().view(torch.float32).double()) / 64
        codes, scales = _block_pool(s)["codes"].double().contiguous(), _block_pool(s)["scales"].double().contiguous()
        f = s["fresh"].long()
        m32 = means[f].float()
        scales.view(-1)[f] = (m32.abs().amax(1) / 448).double()
        codes.view(-1, 128)[f] = (m32 / (m32.abs().amax(1) / 448)[:, None]).to(E4M3).double()
        held = codes.view(-1, 128) * scales.view(-1)[:, None]
        q8 = s["iq8"].view(E4M3).double() * s["iq_scale"].double()[:, None, None]
        for t, (r, n) in enumerate(_visible(case)):
            nb = (n - 1) // 64
            if nb:
                kb = held[s["table"][r, :nb].long()]
                c = 0.4 * math.log(n) if case["ssmax"] else 1.0
                scores[t, :nb] = c * (s["iw"][t].double() @ torch.relu(q8[t] @ kb.T))
        return {"codes": codes, "scales": scales, "scores": scores}
    out, lse = [], []
    blocks = torch.full((s["tokens"], case.get("blocks", 1)), -1, dtype=torch.int32)
    count = torch.zeros(s["tokens"], dtype=torch.int32)
    span = torch.arange(64, device="cuda")
    for t, (r, n) in enumerate(_visible(case)):
        if case["op"] == "paged":
            first = max(0, n - case["window"]) if case["window"] else 0
            where = torch.arange(first, n, device="cuda")
        else:
            row = s["scores"][t, :(n - 1) // 64].cpu()
            picks = sorted(sorted(range(len(row)), key=row.neg().tolist().__getitem__)[:case["blocks"] - 1]) + [(n - 1) // 64]
            blocks[t, :len(picks)] = torch.tensor(picks, dtype=torch.int32)
            count[t] = len(picks)
            where = (torch.tensor(picks, device="cuda")[:, None] * 64 + span).flatten()
            where = where[where < n]
        o, l = _exact_token(s, t, s["table"][r].long()[where // 64] * 64 + where % 64, n)
        out.append(o)
        lse.append(l)
    got = {"out": torch.stack(out), "lse": torch.stack(lse)}
    return got if case["op"] == "paged" else {"blocks": blocks, "blocks_len": count, **got}
