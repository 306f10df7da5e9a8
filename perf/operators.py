"""Measured cases of the 8-bit KV cache and of the cache's pages.

Operators: appending K and V tokens to a paged cache held in e4m3 with one
power-of-two scale per block of tokens and head ("append"); sparse GQA
attention over that cache, one query token per sequence ("decode") or several
("prefill"); and the cache's pages: copying them ("copy"), forking sequences
("fork"), freeing sequences and giving their room to others ("turn"), and
compacting the pool ("compact").

Where ``own`` is false ``run`` computes the operators with elementary torch
operations in 32 bits; where it is true it calls the library.  Outputs held
in 8 bits are returned as e4m3 or e8m0 tensors, that is as values.
"""
import math

import torch

own = False

PAGE = 64        # tokens per cache page
E4M3_MAX = 448.0
EXP_LO, EXP_HI = 87, 167   # scale bytes that the cache holds: 2^-40 .. 2^40
F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu

_LAYER = dict(Hq=32, Hkv=4, D=128, dI=64, k=2048, block=64)   # the layer of the prefill and decode workloads
_TINY = dict(Hq=8, Hkv=2, D=64, dI=32, k=64, block=16)        # the tiny layer


def listed():
    return [
        # one new token for each sequence of a decode batch: latency counts
        dict(name="append-decode-32", op="append", seqs=32, new_lo=1, new_hi=1, len_lo=1000, len_hi=8000, **_LAYER),
        # a 32K prompt written into an empty cache
        dict(name="append-prompt-32k", op="append", seqs=1, new_lo=32768, new_hi=32768, len_lo=0, len_hi=0, **_LAYER),
        # decode of one long sequence: the smallest call of serving
        dict(name="decode-1", op="decode", seqs=1, len_lo=131072, len_hi=131072, **_LAYER),
        # the batch-32 decode workload, cached lengths 32K to 256K
        dict(name="decode-32", op="decode", seqs=32, len_lo=32768, len_hi=262144, **_LAYER),
        # a wide batch of short sequences, some below the budget: rows padded with -1, head dim 64
        dict(name="decode-200-short", op="decode", seqs=200, len_lo=1, len_hi=4100, Hq=16, Hkv=2, D=64, dI=32, k=512,
             block=32),
        # a chunk of a long prompt over the part that is cached already
        dict(name="prefill-chunk-2k", op="prefill", seqs=1, new_lo=2048, new_hi=2048, len_lo=30720, len_hi=30720,
             **_LAYER),
        # a few tokens for each of several sequences (drafted tokens being checked)
        dict(name="prefill-drafts", op="prefill", seqs=9, new_lo=1, new_hi=8, len_lo=500, len_hi=20001, **_LAYER),
        # pages of a long prefix copied to a sequence of its own
        dict(name="copy-2048", op="copy", seqs=4, len_lo=32768, len_hi=32768, pairs=2048, **_LAYER),
        # several samples of each prompt: earlier ones are dropped, new ones forked
        dict(name="fork-64", op="fork", seqs=8, each=8, len_lo=2000, len_hi=9000, **_LAYER),
        # one beam step of a small model
        dict(name="fork-beam-4", op="fork", seqs=1, each=4, len_lo=300, len_hi=300, **_TINY),
        # a batch's sequences leave and others take their slots
        dict(name="turn-32", op="turn", seqs=48, each=32, len_lo=500, len_hi=30000, **_LAYER),
        # a fragmented pool brought together
        dict(name="compact", op="compact", seqs=24, len_lo=500, len_hi=9000, holes=0.4, **_LAYER),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "copy", "fork", "turn", "compact"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, Hq=Hkv * rng.choice([1, 2, 5, 7, 8]), Hkv=Hkv, D=D, dI=rng.choice([32, 64, 128]),
             k=_log(rng, 16, 2048), block=rng.choice([16, 32, 64]))
    if op == "append":
        c["seqs"] = _log(rng, 1, 100)
        if rng.random() < 0.5:
            c.update(new_lo=1, new_hi=1, len_lo=rng.randint(0, 500), len_hi=_log(rng, 501, 8000))
        else:
            most = _log(rng, 2, max(2, 60000 // (c["seqs"] * Hkv * D // 128 + 1)))
            c.update(new_lo=rng.randint(1, most), new_hi=most, len_lo=0, len_hi=rng.choice([0, 63, 3001]))
    elif op == "decode":
        c["seqs"] = _log(rng, 1, 300)
        hi = _log(rng, 10, max(20, min(262144, 3000000 // c["seqs"])))
        c.update(len_lo=rng.randint(1, hi), len_hi=hi)
    elif op == "prefill":
        c["seqs"] = rng.randint(1, 12)
        most = _log(rng, 2, max(2, 1500 // c["seqs"]))
        lo = rng.choice([0, 1, 1000])
        c.update(new_lo=rng.randint(1, most), new_hi=most, len_lo=lo, len_hi=lo + _log(rng, 10, 12000))
    elif op == "copy":
        c.update(seqs=1, len_lo=64, len_hi=64, pairs=_log(rng, 1, 2000 * 512 // max(512, Hkv * D)))
    else:
        c["seqs"] = _log(rng, 1, 40)
        hi = _log(rng, 70, 6000)
        c.update(len_lo=rng.randint(1, hi), len_hi=hi)
        if op == "fork":
            c["each"] = rng.randint(1, 8)
        elif op == "turn":
            c["each"] = rng.randint(1, c["seqs"])
        else:
            c["holes"] = round(rng.uniform(0.0, 0.9), 3)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _scale_bytes(amax):
    """The scale byte of a block: the least e with amax <= 448 * 2^(e - 127), within the cache's range."""
    m, x = torch.frexp(amax)
    return (x - 9 + (m > 0.875).to(x.dtype) + 127).clamp(EXP_LO, EXP_HI)


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _filled(pages, c, gen, spread):
    """A pool's K or V: e4m3 bytes [pages, 64, Hkv, D] and scale bytes [pages, 64 / block, Hkv] of normal values
    with the channels' own spreads, made 2048 pages at a time."""
    data = torch.empty(pages, PAGE, c["Hkv"], c["D"], dtype=torch.uint8, device="cuda")
    exps = torch.empty(pages, PAGE // c["block"], c["Hkv"], dtype=torch.uint8, device="cuda")
    for p0 in range(0, pages, 2048):
        n = min(2048, pages - p0)
        x = torch.randn(n, PAGE // c["block"], c["block"], c["Hkv"], c["D"], generator=gen, device="cuda") * spread
        e = _scale_bytes(x.abs().amax(dim=(2, 4)))
        data[p0:p0 + n] = (x * _pow2(127 - e)[:, :, None, :, None]).to(F8).view(torch.uint8).view_as(data[p0:p0 + n])
        exps[p0:p0 + n] = e.to(torch.uint8)
    return data, exps


def _pool(c, gen, pages):
    spread = torch.exp(0.5 * torch.randn(c["Hkv"], c["D"], generator=gen, device="cuda"))
    k, ek = _filled(pages, c, gen, spread)
    v, ev = _filled(pages, c, gen, 1.0)
    return dict(k=k, v=v, exp=torch.stack([ek, ev], dim=-1).contiguous())


def _keys(c, gen, pages):
    """The indexer's keys of a pool."""
    return dict(k8=torch.randn(pages, PAGE, c["dI"], generator=gen, device="cuda").mul_(100).to(F8).view(torch.uint8),
                ks=torch.rand(pages, PAGE, generator=gen, device="cuda") + 0.5)


def _lengths(lo, hi, n, cpu):
    """n lengths spread evenly over lo .. hi, in random order: their sum goes by the case alone."""
    if n == 1:
        return torch.tensor([hi])
    return (lo + (hi - lo) * torch.arange(n, dtype=torch.float64) / (n - 1)).long()[torch.randperm(n, generator=cpu)]


def _pages(lens):
    return (lens + PAGE - 1) // PAGE


def _deal(lens, pages, rows, most, cpu):
    """Block table [rows, most] of sequences of `lens` tokens on randomly dealt pages."""
    need = _pages(lens)
    table = torch.full((rows, most), -1, dtype=torch.int32)
    at = torch.arange(most)[None, :] < need[:, None]
    table[: len(lens)][at] = torch.randperm(pages, generator=cpu)[: int(need.sum())].to(torch.int32)
    return table


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    op, n = c["op"], c["seqs"]
    s = dict(case=c, sm_scale=1.0 / math.sqrt(c["D"]))
    if op in ("append", "decode", "prefill"):
        old = _lengths(c["len_lo"], c["len_hi"], n, cpu)
        new = _lengths(c.get("new_lo", 0), c.get("new_hi", 0), n, cpu)
        lens = old + new
        pages = int((_pages(old) + _pages(new)).sum()) + 3
        s.update(_pool(c, gen, pages))
        s["table"] = _deal(lens, pages, n, max(1, int(_pages(old.max() + new.max()))), cpu).cuda()
        s["lens"] = lens.to(torch.int32).cuda()
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
        s["cu"] = cu.to(torch.int32).cuda()
        rows = int(cu[-1])
    if op == "append":
        s.update(_keys(c, gen, pages))
        s["single"] = c["new_hi"] == 1
        # K and V as a fused projection leaves them: parts of one row per token
        wide = torch.randn(rows, 2, c["Hkv"], c["D"], generator=gen, device="cuda")
        wide *= 1.0 + torch.rand(rows, 1, 1, 1, generator=gen, device="cuda")
        s["qkv"] = torch.cat([torch.zeros(rows, c["Hq"] * c["D"], device="cuda"), wide.flatten(1)], 1).to(torch.bfloat16)
        at = c["Hq"] * c["D"]
        s["K"] = s["qkv"][:, at:at + c["Hkv"] * c["D"]].unflatten(1, (c["Hkv"], c["D"]))
        s["V"] = s["qkv"][:, at + c["Hkv"] * c["D"]:].unflatten(1, (c["Hkv"], c["D"]))
        s["k8_new"] = torch.randn(rows, c["dI"], generator=gen, device="cuda").mul_(100).to(F8).view(torch.uint8)
        s["ks_new"] = torch.rand(rows, generator=gen, device="cuda") + 0.5
    elif op in ("decode", "prefill"):
        if op == "decode":
            seen = s["lens"].to(torch.int64)
        else:
            of = torch.repeat_interleave(torch.arange(n), new)
            seen = (old[of] + torch.arange(rows) - cu[of] + 1).cuda()
        s["rows"] = rows = len(seen)
        s["q"] = torch.randn(rows, c["Hq"], c["D"], generator=gen, device="cuda").to(torch.bfloat16)
        s["idx"] = torch.full((rows, c["k"]), -1, dtype=torch.int32, device="cuda")
        for r0 in range(0, rows, 256):  # distinct positions of 0 .. seen-1, ascending, padded with -1
            m = seen[r0:r0 + 256]
            width = max(int(m.max()), 1)
            x = torch.rand(len(m), width, generator=gen, device="cuda")
            x.masked_fill_(torch.arange(width, device="cuda")[None, :] >= m[:, None], -1.0)
            top, at = x.topk(min(c["k"], width), dim=1)
            at = torch.where(top >= 0, at, width).sort(dim=1).values
            s["idx"][r0:r0 + 256, : at.shape[1]] = torch.where(at < width, at, -1).to(torch.int32)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, c["Hq"], device="cuda")
    elif op == "copy":
        pages = 2 * c["pairs"] + 5
        s.update(_pool(c, gen, pages))
        s.update(_keys(c, gen, pages))
        both = torch.randperm(pages, generator=cpu)[: 2 * c["pairs"]].to(torch.int32)
        s["src"], s["dst"] = both[: c["pairs"]].cuda(), both[c["pairs"]:].cuda()
    else:
        lens = _lengths(c["len_lo"], c["len_hi"], n, cpu)
        held = int(_pages(lens).sum())
        slots = n
        if op == "fork":
            slots, pages = n * (1 + c["each"]), held + n * c["each"] + 2
        elif op == "turn":
            pages = held + held // 8 + 2
        else:
            pages = max(held, int(held / (1.0 - c["holes"])))
        s["table"] = _deal(lens, pages, slots, max(1, int(_pages(lens.max()))), cpu).cuda()
        s["refs"] = torch.zeros(pages, dtype=torch.int32)
        s["refs"][s["table"].cpu()[s["table"].cpu() >= 0].long()] = 1
        s["refs"] = s["refs"].cuda()
        s["lens"] = torch.cat([lens, torch.zeros(slots - n, dtype=torch.int64)]).to(torch.int32).cuda()
        if op != "turn":
            s.update(_pool(c, gen, pages))
            s.update(_keys(c, gen, pages))
        if op == "fork":
            s["parents"] = torch.arange(n).repeat_interleave(c["each"]).to(torch.int32).cuda()
            s["children"] = (n + torch.randperm(n * c["each"], generator=cpu)).to(torch.int32).cuda()
            s["status"] = torch.empty(n * c["each"], dtype=torch.int32, device="cuda")
        elif op == "turn":
            s["slots"] = torch.randperm(n, generator=cpu)[: c["each"]].to(torch.int32).cuda()
            most = s["table"].shape[1] * PAGE
            s["new_lens"] = _lengths(c["len_lo"], min(c["len_hi"], most), c["each"], cpu).to(torch.int32).cuda()
            s["status"] = torch.empty(c["each"], dtype=torch.int32, device="cuda")
        else:
            s["table_out"] = torch.empty_like(s["table"])
            s["refs_out"] = torch.empty_like(s["refs"])
            s["map"] = torch.empty_like(s["refs"])
            s["used"] = torch.empty(1, dtype=torch.int32, device="cuda")
            s["ws"] = torch.empty(pages * 4 + 64, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the operators in their plain form
# ---------------------------------------------------------------------------

def _places(s):
    """Page, slot and sequence of each token or query row of packed sequences."""
    cu, lens = s["cu"].long(), s["lens"].long()
    new = cu[1:] - cu[:-1]
    of = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), new)
    pos = lens[of] - new[of] + torch.arange(len(of), device="cuda") - cu[of]
    return of, pos


def _append(s):
    c = s["case"]
    block, per = c["block"], PAGE // c["block"]
    of, pos = _places(s)
    page = s["table"][of, pos // PAGE].long()
    slot = pos % PAGE
    at = page * per + slot // block                       # each token's block
    blocks, which = torch.unique(at, return_inverse=True)
    first = torch.full((len(blocks),), block, device="cuda").scatter_reduce(0, which, slot % block, "amin")
    old = s["exp"].view(-1, c["Hkv"], 2)[blocks].int()    # [blocks, Hkv, 2]
    old = torch.where((first > 0)[:, None, None], old, EXP_LO)
    x = torch.stack([s["K"], s["V"]], -1).float()         # [tokens, Hkv, D, 2]
    amax = torch.zeros(len(blocks), c["Hkv"], 2, device="cuda").index_reduce(0, which, x.abs().amax(2), "amax")
    e = torch.maximum(_scale_bytes(amax), old)
    s["exp"].view(-1, c["Hkv"], 2)[blocks] = e.to(torch.uint8)
    kept = torch.arange(block, device="cuda")[None, :] < first[:, None]
    for i, name in enumerate(("k", "v")):
        rows = s[name].view(-1, block, c["Hkv"], c["D"])
        was = rows[blocks]
        y = was.view(F8).float() * _pow2(old[..., i] - e[..., i])[:, None, :, None]
        rows[blocks] = torch.where(kept[:, :, None, None], y.to(F8).view(torch.uint8), was)
        y = (x[..., i] * _pow2(127 - e[..., i])[which][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        s[name].view(-1, c["Hkv"], c["D"])[page * PAGE + slot] = y.to(F8).view(torch.uint8)
    s["k8"].view(-1, c["dI"])[page * PAGE + slot] = s["k8_new"]
    s["ks"].view(-1)[page * PAGE + slot] = s["ks_new"]


def _attend(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "decode":
        of, pos = torch.arange(s["rows"], device="cuda"), s["lens"].long() - 1
    else:
        of, pos = _places(s)
    idx = s["idx"].long()
    ok = (idx >= 0) & (idx <= pos[:, None])
    idx = idx.clamp(min=0)
    page = s["table"][of[:, None], idx // PAGE].long().clamp(min=0)
    at, part = page * PAGE + idx % PAGE, page * (PAGE // c["block"]) + idx % PAGE // c["block"]
    scale = _pow2(s["exp"].view(-1, c["Hkv"], 2)[part].int() - 127)          # [rows, k, Hkv, 2]
    q = s["q"].float().unflatten(1, (c["Hkv"], G))
    K = s["k"].view(F8).view(-1, c["Hkv"], c["D"])[at].float() * scale[..., 0:1]
    x = torch.einsum("rgjd,rkgd->rgjk", q, K) * s["sm_scale"]
    del K
    x = x.masked_fill(~ok[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    V = s["v"].view(F8).view(-1, c["Hkv"], c["D"])[at].float() * scale[..., 1:2]
    o = torch.einsum("rgjk,rkgd->rgjd", p, V) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.flatten(1, 2))
    s["lse"].copy_((top + torch.log(total)).flatten(1))


def _copy(s, src, dst):
    for name in ("k", "v", "exp", "k8", "ks"):
        s[name][dst] = s[name][src]


def _room(table, lens, refs, slots):
    """Takes the pages of the sequences in `slots` off the pool's counts and empties their rows."""
    rows = table[slots]
    used = torch.arange(rows.shape[1], device="cuda")[None, :] < ((lens[slots] + PAGE - 1) // PAGE)[:, None]
    ids = rows[used].long()
    refs.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    table[slots] = -1
    lens[slots] = 0


def _granted(refs, need):
    """Which of the asked counts of pages the pool can give, in order, and the pages: the lowest free ids."""
    free = torch.nonzero(refs == 0).flatten()
    ok = (need == 0) | (need.cumsum(0) <= len(free))
    return ok, free[: int((need * ok).sum())]


def _fork(s):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    par, chi = s["parents"].long(), s["children"].long()
    _room(table, lens, refs, chi)
    n = lens[par].long()
    part = n % PAGE != 0
    ok, got = _granted(refs, part.long())
    par, chi, n, part = par[ok], chi[ok], n[ok], part[ok]
    refs[got] = 1
    full = torch.arange(table.shape[1], device="cuda")[None, :] < (n // PAGE)[:, None]
    table[chi] = torch.where(full, table[par], -1)
    lens[chi] = n.int()
    ids = table[par][full].long()
    refs.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    tail = (n // PAGE)[part]
    src = table[par[part], tail].long()
    table[chi[part], tail] = got.int()
    _copy(s, src, got)
    s["status"].copy_((~ok).int())


def _turn(s):
    table, lens, refs, slots = s["table"], s["lens"], s["refs"], s["slots"].long()
    _room(table, lens, refs, slots)
    need = (s["new_lens"].long() + PAGE - 1) // PAGE
    ok, got = _granted(refs, need)
    refs[got] = 1
    width = torch.arange(table.shape[1], device="cuda")[None, :]
    rows = table[slots]
    rows[width < (need * ok)[:, None]] = got.int()
    table[slots] = rows
    lens[slots] = s["new_lens"] * ok
    s["status"].copy_((~ok).int())


def _compact(s):
    used = s["refs"] != 0
    n = int(used.sum())
    ids = torch.arange(len(used), device="cuda")
    high, low = ids[n:][used[n:]], ids[:n][~used[:n]]
    to = torch.where(used, ids, -1)
    to[high] = low
    s["map"].copy_(to)
    s["used"].fill_(n)
    s["refs_out"].copy_(s["refs"])
    s["refs_out"][low] = s["refs"][high]
    s["refs_out"][n:] = 0
    held = torch.arange(s["table"].shape[1], device="cuda")[None, :] < ((s["lens"] + PAGE - 1) // PAGE)[:, None]
    s["table_out"].copy_(torch.where(held, to[s["table"].clamp(min=0)], -1))
    _copy(s, high, low)


def _own(s):
    from sparse_long_context_03_b200 import dsa
    c, op = s["case"], s["case"]["op"]
    if op == "append":
        dsa.kv8_append(s["K"], s["V"], s["k"], s["v"], s["exp"], s["table"], s["lens"],
                       cu_seqlens=None if s["single"] else s["cu"], k8=s["k8_new"], k_scale=s["ks_new"],
                       k8_cache=s["k8"], k_scale_cache=s["ks"])
    elif op == "decode":
        dsa.sparse_gqa_decode_attention_kv8(s["q"], s["k"], s["v"], s["exp"], s["table"], s["lens"], s["idx"],
                                            c["k"], s["sm_scale"], s["out"], s["lse"])
    elif op == "prefill":
        dsa.sparse_gqa_prefill_kv8(s["q"], s["k"], s["v"], s["exp"], s["table"], s["lens"], s["idx"], s["cu"], 0,
                                   s["rows"], c["k"], s["sm_scale"], s["out"], s["lse"])
    elif op == "turn":
        dsa.pages_free(s["slots"], s["table"], s["lens"], s["refs"])
        dsa.pages_extend(s["slots"], s["new_lens"], s["table"], s["lens"], s["refs"], s["status"])
    else:
        bufs = [s["k"], s["v"], s["exp"], s["k8"], s["ks"]]
        if op == "copy":
            dsa.pages_copy(bufs, s["src"], s["dst"])
        elif op == "fork":
            dsa.pages_free(s["children"], s["table"], s["lens"], s["refs"])
            dsa.pages_fork(bufs, s["parents"], s["children"], s["table"], s["lens"], s["refs"], s["status"])
        else:
            dsa.pages_compact(bufs, s["table"], s["lens"], s["refs"], s["map"], s["used"], s["ws"],
                              block_table_out=s["table_out"], refcount_out=s["refs_out"])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        _own(s)
    elif op == "append":
        _append(s)
    elif op in ("decode", "prefill"):
        _attend(s)
    elif op == "copy":
        _copy(s, s["src"].long(), s["dst"].long())
    elif op == "fork":
        _fork(s)
    elif op == "turn":
        _turn(s)
    else:
        _compact(s)
    if op in ("decode", "prefill"):
        return dict(out=s["out"], lse=s["lse"])
    got = {}
    if op != "turn":
        got.update(k=s["k"].view(F8), v=s["v"].view(F8), scale=s["exp"].view(E8), k8=s["k8"].view(F8), ks=s["ks"])
    if op in ("fork", "turn"):
        got.update(table=s["table"], lens=s["lens"], refs=s["refs"], status=s["status"])
    elif op == "compact":
        got.update(table=s["table_out"], refs=s["refs_out"], map=s["map"], used=s["used"])
    return got


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    n, mean = c["seqs"], (c["len_lo"] + c["len_hi"]) / 2
    token = 2 * c["Hkv"] * c["D"]                         # bytes of a cached token's K and V
    page = PAGE * (token + c["dI"] + 4) + 2 * c["Hkv"] * PAGE // c["block"]
    if op == "append":
        rows = n * (c["new_lo"] + c["new_hi"]) / 2
        return {"bytes": rows * (3 * token + 2 * (c["dI"] + 4)), "flops": rows * token * 3}
    if op in ("decode", "prefill"):
        new = (c["new_lo"] + c["new_hi"]) / 2 if op == "prefill" else 1
        rows, sees = n * new, min(c["k"], mean + (new + 1) / 2 if op == "prefill" else mean)
        read = min(rows * sees, n * (mean + new)) * (token + 2 * c["Hkv"] / c["block"])
        return {"bytes": read + rows * (c["Hq"] * (4 * c["D"] + 4) + 4 * sees),
                "flops": 4 * rows * sees * c["Hq"] * c["D"]}
    held = n * (mean + PAGE / 2) / PAGE
    if op == "copy":
        return {"bytes": c["pairs"] * (2 * page + 8), "flops": 0}
    if op == "fork":
        return {"bytes": n * c["each"] * (2 * page + (mean / PAGE) * 16), "flops": 0}
    if op == "turn":
        return {"bytes": c["each"] * (mean / PAGE + 1) * 20, "flops": 0}
    moved = held * c["holes"]
    return {"bytes": moved * 2 * page + held * 20, "flops": 0}


def _e4m3_values(data):
    """The values of e4m3 bytes in 64 bits, from the format: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    b = torch.arange(256, device="cuda")
    e, m = ((b >> 3) & 15).double(), (b & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    return torch.where(b >= 128, -v, v)[data.long()]


def _to_e4m3(y):
    """The nearest e4m3 value, ties to the even one, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(s):
    c = s["case"]
    block, lens, cu, table = c["block"], s["lens"].tolist(), s["cu"].tolist(), s["table"].tolist()
    vals = {"k": _e4m3_values(s["k"]), "v": _e4m3_values(s["v"])}
    k8, ks, exps = _e4m3_values(s["k8"]), s["ks"].double(), s["exp"].double() - 127
    new8 = _e4m3_values(s["k8_new"])
    for b in range(len(lens)):
        t, pos = cu[b], lens[b] - (cu[b + 1] - cu[b])
        while t < cu[b + 1]:  # the tokens that go to one block
            at, page = pos % block, table[b][pos // PAGE]
            m = min(block - at, cu[b + 1] - t)
            lo, part = pos % PAGE, pos % PAGE // block
            for i, (name, src) in enumerate((("k", "K"), ("v", "V"))):
                x = s[src][t:t + m].double()
                all_e = torch.arange(EXP_LO - 127.0, EXP_HI - 126.0, device="cuda", dtype=torch.float64)
                fits = x.abs().amax((0, 2))[:, None] <= E4M3_MAX * torch.exp2(all_e)[None, :]
                fits[:, -1] = True
                e = all_e[fits.long().argmax(1)]
                was = exps[page, part, :, i].clone()
                if at:
                    e = torch.maximum(e, was)
                    kept = vals[name][page, lo - at:lo]
                    vals[name][page, lo - at:lo] = _to_e4m3(kept * torch.exp2(was - e)[None, :, None])
                vals[name][page, lo:lo + m] = _to_e4m3(x * torch.exp2(-e)[None, :, None])
                exps[page, part, :, i] = e
            k8[page, lo:lo + m] = new8[t:t + m]
            ks[page, lo:lo + m] = s["ks_new"][t:t + m].double()
            t, pos = t + m, pos + m
    return dict(k=vals["k"], v=vals["v"], scale=torch.exp2(exps), k8=k8, ks=ks)


def _exact_attend(s):
    c = s["case"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["rows"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    K, V = (s[n].view(-1, c["Hkv"], c["D"]) for n in ("k", "v"))
    for b in range(len(lens)):
        rows = range(b, b + 1) if c["op"] == "decode" else range(cu[b], cu[b + 1])
        for r in rows:
            last = lens[b] - len(rows) + (r - rows[0])
            i = s["idx"][r].long()
            i = i[(i >= 0) & (i <= last)]
            if not len(i):
                continue
            page = s["table"][b, i // PAGE].long()
            at = page * PAGE + i % PAGE
            e = torch.exp2(s["exp"][page, i % PAGE // c["block"]].double() - 127)     # [n, Hkv, 2]
            q = s["q"][r].double().view(c["Hkv"], -1, c["D"])
            x = q @ (_e4m3_values(K[at]) * e[..., :1]).permute(1, 2, 0) / math.sqrt(c["D"])
            lse[r] = torch.logsumexp(x, -1).flatten()
            out[r] = (torch.softmax(x, -1) @ (_e4m3_values(V[at]) * e[..., 1:]).transpose(0, 1)).flatten(0, 1)
    return dict(out=out, lse=lse)


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    if case["op"] in ("decode", "prefill"):
        return _exact_attend(prepare(case, seed))
    return None  # pages are moved and counted: nothing is computed that could be off
