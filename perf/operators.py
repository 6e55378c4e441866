"""The cache operators of a serving step, with cases to time and compare them.

Two operators over a paged cache of keys and values:

- "write": new tokens' keys and values into the cache's pages (8 bits with a
  power-of-two scale per page and head, or bf16), the position rotation applied
  to the keys, and to the step's queries, on the way;
- "attn": exact softmax attention over rows of selected tokens, read from the
  pages.

`run` computes them in elementary torch operations, or with the framework's
calls where `own` is set.  Layouts: new K, V [tokens][hkv][d]; pages
[n_pages][hkv][page][d]; scales [n_pages][hkv]; page table [batch][ld_pages];
selection rows [batch][nq][hkv][max_sel].
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}
#: largest magnitude under scale 1: e4m3's largest value for V; for K 316, since a
#: rotation makes a component at most sqrt(2) larger and 316 * sqrt(2) < 448
LIM_K, LIM_V = 316.0, 448.0
#: scales are powers of two between these exponents
EXP_MIN, EXP_MAX = -64, 64


def listed():
    return [
        # one decode step of four sequences near 10M tokens: four tokens, nothing but latency
        write_case("write_decode_4", batch=4, new=1, start=10_000_003, hq=16, hkv=1, d=128, page=64, cache="e4m3"),
        # a decode step of many users, positions anywhere in their pages
        write_case("write_decode_96", batch=96, new=1, start=30_011, hq=32, hkv=4, d=128, page=32, cache="e4m3"),
        # a mixed step: ragged chunks of several prompts, half the dimensions rotated, pairs interleaved, bf16 pages
        write_case("write_chunks_ragged", batch=7, new=700, start=1_017, hq=12, hkv=4, d=64, page=16, cache="bf16",
                   rot=32, interleaved=True, ragged=True),
        # a long prompt's chunk, fp32 activations
        write_case("write_chunk_f32", batch=1, new=8191, start=65_541, hq=8, hkv=2, d=128, page=128, cache="e4m3",
                   io="f32"),
        # a whole prompt of 128K tokens, 32 query and 4 KV heads
        write_case("write_prompt_128k", batch=1, new=131_072, start=0, hq=32, hkv=4, d=128, page=64, cache="e4m3"),
        # speculative decoding: a few queries each over short ragged rows, some of them empty, fp32 in and out
        attn_case("attn_short_f32", batch=3, nq=5, ctx=401, hq=12, hkv=4, d=64, page=16, cache="e4m3", io="f32",
                  topk=61, pool=1, sink=3, window=13, ragged=True),
        # one decode step of four long sequences, one KV head: top 2,048 + 64 sink + 2,048 window
        attn_case("attn_decode_4", batch=4, nq=1, ctx=1_000_003, hq=16, hkv=1, d=128, page=64, cache="e4m3",
                  topk=2048, pool=4, sink=64, window=2048),
        # ordinary serving: 16 users, bf16 pages, ragged rows
        attn_case("attn_decode_bf16", batch=16, nq=1, ctx=20_011, hq=32, hkv=8, d=64, page=32, cache="bf16",
                  topk=1024, pool=4, sink=64, window=511, ragged=True),
        # a decode step of 96 users, 32 query and 4 KV heads
        attn_case("attn_decode_96", batch=96, nq=1, ctx=30_011, hq=32, hkv=4, d=128, page=32, cache="e4m3",
                  topk=2048, pool=4, sink=64, window=512),
        # the last 65 queries of one prompt, no sharing between heads
        attn_case("attn_chunk_65", batch=1, nq=65, ctx=9_001, hq=4, hkv=4, d=128, page=128, cache="e4m3",
                  topk=1001, pool=3, sink=5, window=300),
        # a prompt's chunk of 2,048 queries over a 128K context, 16 query and 2 KV heads
        attn_case("attn_chunk_2k", batch=1, nq=2048, ctx=131_072, hq=16, hkv=2, d=128, page=64, cache="e4m3",
                  topk=2048, pool=4, sink=64, window=1024),
    ]


def write_case(name=None, *, batch, new, start, hq, hkv, d, page, cache, io="bf16", rot=None, interleaved=False,
               ragged=False):
    """`batch` sequences; sequence b has `start` + 5 b tokens in the cache and brings `new` more (ragged: fewer)."""
    c = dict(op="write", batch=batch, new=new, start=start, hq=hq, hkv=hkv, d=d, page=page, cache=cache, io=io,
             rot=d if rot is None else rot, interleaved=interleaved, ragged=ragged)
    return dict(c, name=name) if name else c


def attn_case(name=None, *, batch, nq, ctx, hq, hkv, d, page, cache, topk, pool, sink, window, io="bf16",
              ragged=False):
    """The last `nq` positions of `batch` contexts of `ctx` tokens, rows of sink + topk (blocks of `pool`) + window."""
    c = dict(op="attn", batch=batch, nq=nq, ctx=ctx, hq=hq, hkv=hkv, d=d, page=page, cache=cache, io=io, topk=topk,
             pool=pool, sink=sink, window=window, ragged=ragged)
    return dict(c, name=name) if name else c


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["e4m3", "e4m3", "bf16"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    ragged = rng.random() < 0.5
    if rng.random() < 0.4:
        batch = _spread(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _spread(rng, 1, 40_000)
        new = max(1, min(new, 4_000_000 // (batch * (hq + 2 * hkv))))
        return write_case(batch=batch, new=new, start=_spread(rng, 1, 10_000_000) - 1, hq=hq, hkv=hkv, d=d, page=page,
                          cache=cache, io=io, rot=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.5,
                          ragged=ragged)
    batch = _spread(rng, 1, 64)
    nq = 1 if rng.random() < 0.5 else _spread(rng, 1, 512)
    topk, pool = _spread(rng, 1, 4096), rng.choice([1, 2, 3, 4, 8])
    sink, window = rng.randint(0, 64), _spread(rng, 1, 2048)
    rows = topk + sink + window
    nq = max(1, min(nq, 6_000_000 // (batch * hkv * rows)))
    if batch * nq * hq * rows * d > 6_000_000_000:
        batch, hq = 1, hkv
    ctx = rows + nq + pool * 2 + _spread(rng, 1, max(1, min(200_000, 40_000_000 // (batch * hkv * d))))
    return attn_case(batch=batch, nq=nq, ctx=ctx, hq=hq, hkv=hkv, d=d, page=page, cache=cache, io=io, topk=topk,
                     pool=pool, sink=sink, window=window, ragged=ragged)


# ------------------------------------------------------------------ sizes
def _lengths(c):
    """New tokens of each sequence of a write (plain arithmetic, no seed): ragged ones fall to a few, or to none."""
    if not c["ragged"]:
        return [c["new"]] * c["batch"]
    return [0 if b % 5 == 2 else max(1, (c["new"] * (1 + (7 * b) % 11)) // 11) for b in range(c["batch"])]


def _counts(c):
    """Length of every selection row [batch][nq][hkv] (plain arithmetic, no seed)."""
    full = c["sink"] + c["topk"] + c["window"]
    n = c["batch"] * c["nq"] * c["hkv"]
    i = torch.arange(n, dtype=torch.int64)
    if c["ragged"]:
        cnt = 1 + (i * 2654435761 + 12345) % (1 << 20) * full // (1 << 20)
        cnt[i % 11 == 3] = 0
        cnt[i % 11 == 5] = full
    else:
        cnt = torch.full((n,), full, dtype=torch.int64)
    return cnt.view(c["batch"], c["nq"], c["hkv"])


def work(case):
    c = case
    io, ce = BYTES[c["io"]], BYTES[c["cache"]]
    if c["op"] == "write":
        n = sum(_lengths(c))
        per = (c["hq"] + 2 * c["hkv"]) * io + (c["hq"] + c["hkv"]) * io + 2 * c["hkv"] * ce
        return {"bytes": n * per * c["d"], "flops": 3 * n * (c["hq"] + c["hkv"]) * c["rot"]}
    cnt = _counts(c)
    rows = int(cnt.sum())
    union = int(torch.clamp(cnt.sum(1), max=c["ctx"]).sum())   # rows that several queries share are read once
    nbytes = union * 2 * c["d"] * ce + rows * 4 + 2 * c["batch"] * c["nq"] * c["hq"] * c["d"] * io
    return {"bytes": nbytes, "flops": 4 * rows * (c["hq"] // c["hkv"]) * c["d"]}


# ----------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _heads(g, n, h, d, dtype):
    """Activations [n][h][d]: per-channel spreads, a few strong channels, as projected keys and queries have."""
    chan = torch.exp(0.4 * _normal(g, h, d))
    chan[:, 3] *= 8.0
    return (_normal(g, n, h, d) * chan).to(dtype)


def _filled_pages(g, n_pages, c, lim):
    """Pages full of tokens, and their scales as _scale says (None for bf16 pages)."""
    dt = TYPES[c["cache"]]
    x = _heads(g, n_pages * c["page"], c["hkv"], c["d"], torch.bfloat16)
    x = x.view(n_pages, c["page"], c["hkv"], c["d"]).transpose(1, 2)
    if c["cache"] != "e4m3":
        return x.contiguous(), None
    s = _scale(x.float().abs().amax((2, 3)), lim)
    return (x.float() / s[:, :, None, None]).to(dt).contiguous(), s


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    io = TYPES[c["io"]]
    s = {"case": c}
    B, page = c["batch"], c["page"]
    if c["op"] == "write":
        lens = torch.tensor(_lengths(c), dtype=torch.int64)
        n = int(lens.sum())
        start = c["start"] + 5 * torch.arange(B)
        last = (start + lens + page - 1) // page              # pages a sequence has after the write
        first = start // page                                 # the earlier ones are not touched: left out of the pool
        n_pages = int((last - first).sum()) + 3
        order = torch.randperm(n_pages, generator=g, device=DEV).cpu()
        table = torch.full((B, int(last.max()) + 1), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            k = int(last[b] - first[b])
            table[b, int(first[b]):int(last[b])] = order[at:at + k].int()
            at += k
        s["K_pages"], s["K_scale"] = _filled_pages(g, n_pages, c, LIM_K)
        s["V_pages"], s["V_scale"] = _filled_pages(g, n_pages, c, LIM_V)
        s["table"] = table.to(DEV)
        pad = 3 if c["ragged"] else 0                         # rows behind the last sequence: not to be written
        s["K"] = _heads(g, n + pad, c["hkv"], c["d"], io)
        s["V"] = _heads(g, n + pad, c["hkv"], c["d"], io)
        s["Q"] = _heads(g, n + pad, c["hq"], c["d"], io)
        s["Q_out"], s["K_out"] = torch.zeros_like(s["Q"]), torch.zeros_like(s["K"])
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(DEV)
        s["pos0"] = start.to(DEV)
        s["inv_freq"] = 10000.0 ** (-torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV) / (c["rot"] // 2))
        return s
    ctx, nq, hkv, P = c["ctx"], c["nq"], c["hkv"], c["pool"]
    per = -(-ctx // page)
    s["K_pages"], s["K_scale"] = _filled_pages(g, B * per, c, LIM_K)
    s["V_pages"], s["V_scale"] = _filled_pages(g, B * per, c, LIM_V)
    s["table"] = torch.randperm(B * per, generator=g, device=DEV).to(torch.int32).view(B, per)
    s["Q"] = _heads(g, B * nq, c["hq"], c["d"], io).view(B, nq, c["hq"], c["d"])
    # selection rows: sink, blocks of P tokens spread over the rest, window; ascending
    cnt = _counts(c).to(DEV)[..., None]
    S, W = c["sink"], c["window"]
    j = torch.arange(S + c["topk"] + W, device=DEV)
    i = (ctx - nq + torch.arange(nq, device=DEV)).view(1, nq, 1, 1)
    s0 = cnt.clamp(max=S)
    w0 = (cnt - s0).clamp(max=W)
    mid = cnt - s0 - w0
    nblk = (mid + P - 1) // P
    total = (i - W + 1 - S) // P                              # blocks between sink and window
    m = (j - s0).clamp(min=0)
    blk = m // P
    u = torch.rand(B, nq, hkv, -(-c["topk"] // P) + 1, generator=g, device=DEV, dtype=torch.float64)
    u = torch.gather(u, 3, blk.clamp(max=u.shape[3] - 1).expand(B, nq, hkv, -1))
    far = S + P * torch.floor((blk + 0.999 * u) * total / nblk.clamp(min=1)).long() + m % P
    tok = torch.where(j < s0, j, torch.where(j >= cnt - w0, i - (cnt - 1 - j), far))
    s["idx"] = torch.where(j < cnt, tok, -1).to(torch.int32).contiguous()
    s["cnt"] = cnt[..., 0].to(torch.int32).contiguous()
    s["O"] = torch.empty_like(s["Q"])
    s["lse"] = torch.empty(B, nq, c["hq"], device=DEV)
    return s


# -------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return _write(state) if state["case"]["op"] == "write" else _attend(state)


def _run_own(s):
    from hierarchical_latent_key_gemm_b200 import lsa
    cache = lsa.KVCache(s["K_pages"], s["V_pages"], s["table"], s["K_scale"], s["V_scale"])
    if s["case"]["op"] == "write":
        lsa.lsa_cache_write(cache, s["K"], s["V"], s["cu"], s["pos0"], Q=s["Q"], inv_freq=s["inv_freq"],
                            interleaved=s["case"]["interleaved"], K_out=s["K_out"], Q_out=s["Q_out"])
        return _written(s)
    O, lse = lsa.lsa_cache_attn(cache, s["Q"], s["idx"], s["cnt"], O=s["O"], lse=s["lse"])
    return {"O": O, "lse": lse}


def _written(s):
    out = {"K_pages": s["K_pages"], "V_pages": s["V_pages"], "Q_out": s["Q_out"], "K_out": s["K_out"]}
    if s["K_scale"] is not None:
        out.update(K_scale=s["K_scale"], V_scale=s["V_scale"])
    return out


def _scale(amax, lim):
    """The smallest power of two 2^e with amax <= lim * 2^e, e between EXP_MIN and EXP_MAX."""
    m, e = torch.frexp(amax)                                  # amax = m * 2^e, m in [0.5, 1)
    lm, le = math.frexp(lim)
    e = e - le + (m > lm).int()
    e = torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)
    return ((e + 127) << 23).view(torch.float32)              # 2^e by its bits


def _rotate(x, cos, sin, rot, interleaved):
    """x [n][h][d], cos and sin [n][rot/2]: the first `rot` components turned pair by pair."""
    y = x.clone()
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def _write(s):
    c = s["case"]
    page = c["page"]
    n = int(sum(_lengths(c)))
    tok = torch.arange(n, device=DEV)
    b = torch.searchsorted(s["cu"], tok, right=True) - 1
    pos = s["pos0"][b] + tok - s["cu"][b]
    pid = s["table"][b, pos // page].long()
    slot = pos % page
    ang = pos[:, None].double() * s["inv_freq"]               # far positions: the angle needs 64 bits
    cos, sin = ang.cos().float(), ang.sin().float()
    k = _rotate(s["K"][:n].float(), cos, sin, c["rot"], c["interleaved"])
    s["Q_out"][:n] = _rotate(s["Q"][:n].float(), cos, sin, c["rot"], c["interleaved"]).to(s["Q"].dtype)
    s["K_out"][:n] = k.to(s["K"].dtype)
    if c["cache"] != "e4m3":
        s["K_pages"][pid, :, slot] = k.to(s["K_pages"].dtype)
        s["V_pages"][pid, :, slot] = s["V"][:n].to(s["V_pages"].dtype)
        return _written(s)
    at = (pid, slot, _first_slots(s, pid, slot, page))
    _store(s["K_pages"], s["K_scale"], k, s["K"][:n], LIM_K, *at)
    _store(s["V_pages"], s["V_scale"], s["V"][:n].float(), s["V"][:n], LIM_V, *at)
    return _written(s)


def _first_slots(s, pid, slot, page):
    """First slot written in every page of the pool (`page`: none)."""
    none = torch.full((s["K_pages"].shape[0],), page, device=DEV, dtype=torch.int64)
    return none.scatter_reduce(0, pid, slot, "amin")


def _store(pages, scale, new, raw, lim, pid, slot, first):
    """`new` into the slots; what a touched page held below its first new slot is kept under the new scale."""
    page = pages.shape[2]
    touched, kept = (first < page)[:, None], ((first > 0) & (first < page))[:, None]
    amax = torch.zeros_like(scale).scatter_reduce(0, pid[:, None].expand(-1, pages.shape[1]),
                                                  raw.float().abs().amax(2), "amax")
    want = _scale(amax, lim)
    want = torch.where(kept, torch.maximum(want, scale), want)
    again = (pages.float() * torch.where(kept, scale / want, 1.0)[:, :, None, None]).to(pages.dtype)
    move = ((torch.arange(page, device=DEV) < first[:, None]) & kept)[:, None, :, None]
    pages.copy_(torch.where(move, again.view(torch.uint8), pages.view(torch.uint8)).view(pages.dtype))
    scale.copy_(torch.where(touched, want, scale))
    pages.view(torch.uint8)[pid, :, slot] = (new / scale[pid][:, :, None]).to(pages.dtype).view(torch.uint8)


def _rows(s, pages, scale, ok, tok):
    """The selected rows of a pool as fp32 [batch][nq][hkv][max_sel][d]."""
    n_pages, hkv, page, d = pages.shape
    B = tok.shape[0]
    b = torch.arange(B, device=DEV).view(B, 1, 1, 1)
    h = torch.arange(hkv, device=DEV).view(1, 1, hkv, 1)
    pid = s["table"][b, tok // page].long()
    row = (pid * hkv + h) * page + tok % page
    flat = pages.view(-1, d)
    if scale is None:
        return flat[row].float()
    x = flat.view(torch.uint8)[row].view(pages.dtype).float()
    return x.mul_(scale[pid, h][..., None])


def _attend(s):
    c = s["case"]
    B, nq, hq, d = s["Q"].shape
    hkv = c["hkv"]
    ok = torch.arange(s["idx"].shape[3], device=DEV) < s["cnt"][..., None]
    tok = torch.where(ok, s["idx"], 0).long()
    q = s["Q"].float().view(B, nq, hkv, hq // hkv, d)
    x = q @ _rows(s, s["K_pages"], s["K_scale"], ok, tok).transpose(3, 4) * (1.0 / math.sqrt(d))
    x.masked_fill_(~ok[:, :, :, None], -math.inf)
    m = x.amax(4, keepdim=True)
    p = torch.exp(x - m.clamp(min=-1e30))
    total = p.sum(4, keepdim=True)
    o = p @ _rows(s, s["V_pages"], s["V_scale"], ok, tok)
    o = torch.where(total > 0, o / total, 0.0)
    s["O"].copy_(o.view(B, nq, hq, d))
    s["lse"].copy_((m + total.log()).view(B, nq, hq))
    return {"O": s["O"], "lse": s["lse"]}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    def written(s):
        """Every page value before its rounding to the pages' type, token by token of each page."""
        c = s["case"]
        page, n, half = c["page"], int(s["cu"][-1]), c["rot"] // 2
        pos = torch.cat([int(p) + torch.arange(int(s["cu"][b + 1] - s["cu"][b])) for b, p in enumerate(s["pos0"])])
        seq = torch.cat([torch.full((int(s["cu"][b + 1] - s["cu"][b]),), b) for b in range(c["batch"])])
        pos, seq = pos.to(DEV), seq.to(DEV)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           torch.outer(pos.double(), s["inv_freq"]))[:, None]

        def rotated(x):
            x = x.double()
            pairs = x[..., :2 * half]
            pairs = (pairs.unflatten(-1, (half, 2)) if c["interleaved"]
                     else pairs.unflatten(-1, (2, half)).transpose(-1, -2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat([z, x[..., 2 * half:]], -1)

        q, k = s["Q_out"].double(), s["K_out"].double()
        q[:n], k[:n] = rotated(s["Q"][:n]), rotated(s["K"][:n])
        out = {"Q_out": q, "K_out": k}
        pid, slot = s["table"][seq, pos // page].long(), pos % page
        for name, new, raw, lim in (("K", k[:n], s["K"], LIM_K), ("V", s["V"][:n].double(), s["V"], LIM_V)):
            pages, scale = s[name + "_pages"].double(), s[name + "_scale"]
            if scale is None:
                pages[pid, :, slot] = new
            else:
                scale = scale.double()
                big = torch.zeros_like(scale).index_reduce_(0, pid, raw[:n].double().abs().amax(2), "amax")
                low = torch.full((len(scale),), page, device=DEV).index_reduce_(0, pid, slot, "amin")
                powers = torch.tensor([2.0 ** e for e in range(EXP_MIN, EXP_MAX + 1)], dtype=torch.float64, device=DEV)
                want = powers[torch.searchsorted(lim * powers, big).clamp(max=len(powers) - 1)]
                part = ((low > 0) & (low < page))[:, None]
                want = torch.where(part, torch.maximum(want, scale), torch.where((low < page)[:, None], want, scale))
                held = part[:, :, None, None] & (torch.arange(page, device=DEV) < low[:, None])[:, None, :, None]
                pages = torch.where(held, pages * (scale / want)[:, :, None, None], pages)
                pages[pid, :, slot] = new / want[pid][:, :, None]
                out[name + "_scale"] = want
            out[name + "_pages"] = pages
        return out

    def attended(s):
        c = s["case"]
        B, nq, hq, d = s["Q"].shape
        hkv, page, G = c["hkv"], c["page"], hq // c["hkv"]
        O = torch.zeros(B, nq, hq, d, dtype=torch.float64, device=DEV)
        lse = torch.full((B, nq, hq), -math.inf, dtype=torch.float64, device=DEV)
        pools = [(s[n + "_pages"], s[n + "_scale"]) for n in "KV"]
        for b in range(B):
            for h in range(hkv):
                dense = []
                for pages, scale in pools:
                    mine = s["table"][b].long()
                    x = pages.view(torch.uint8)[mine, h].view(pages.dtype).double()
                    dense.append((x if scale is None else x * scale[mine, h].double()[:, None, None]).view(-1, d))
                for q0 in range(0, nq, 64):
                    idx, cnt = s["idx"][b, q0:q0 + 64, h].long(), s["cnt"][b, q0:q0 + 64, h]
                    hole = idx < 0
                    q = s["Q"][b, q0:q0 + 64, h * G:(h + 1) * G].double()
                    x = torch.einsum("qgd,qjd->qgj", q, dense[0][idx.clamp(min=0)]) / d ** 0.5
                    x = x.masked_fill(hole[:, None], -math.inf)
                    z = torch.logsumexp(x, 2)
                    p = torch.where(cnt[:, None, None] > 0, torch.exp(x - z[..., None]), 0.0)
                    O[b, q0:q0 + 64, h * G:(h + 1) * G] = torch.einsum("qgj,qjd->qgd", p, dense[1][idx.clamp(min=0)])
                    lse[b, q0:q0 + 64, h * G:(h + 1) * G] = z
        return {"O": O, "lse": lse}

    s = prepare(case, seed)
    return written(s) if case["op"] == "write" else attended(s)
