"""What is measured of the 4-bit KV cache and of the eviction by accumulated attention weight.

Four operators, each in a plain form (elementary torch operations in fp32) and as the calls of this
library that a user's program makes:

  store   rows of K and V written into a 4-bit cache, the block summary and label slab kept up with
          them, and the rows read back as bf16 (a prompt at once, or one token per sequence);
  attn    attention of one decode step over a 4-bit cache: over the selected tokens, over a slot cache
          of blocks, or over every token;
  weights the softmax weights of a decode step, summed over the heads of each KV head, added to one
          fp32 number per cached token (keys in fp32, bf16, the shared latent, or 4 bits);
  evict   the tokens to keep by that number (the first and the newest always), and the cache's rows
          moved together in place.

The 4-bit cache holds one record of 9 d / 8 bytes per (sequence, KV head, token): d / 2 bytes of K
codes, d / 16 scale bytes of K, d / 16 scale bytes of V, d / 2 bytes of V codes.  A code is an e2m1
number (sign, two exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), channel 2 i in the low
nibble of byte i.  Sixteen channels share a scale byte b: the fp16 number with the bits b << 7.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 64 sequences, in the middle of a block: what every decode step pays
        dict(name="store_append_b64", op="store", batch=64, kv=8, d=128, ctx=4096, old=2021, rows=1, bs=32, r=16),
        # a 48k prompt quantised at once
        dict(name="store_prompt_48k", op="store", batch=1, kv=8, d=128, ctx=49152, old=0, rows=49152, bs=32, r=16),
        # the smallest call: 4 heads on one KV head, 256 tokens; latency only
        dict(name="attn_4k", op="attn", batch=1, kv=1, g=4, d=64, ctx=4096, bs=32, kb=16, kt=256, mode="list",
             ragged=False, out="float32"),
        # one sequence of 48k: few groups, so the tokens of each are split over many SMs
        dict(name="attn_48k", op="attn", batch=1, kv=8, g=4, d=128, ctx=49152, bs=32, kb=192, kt=2048, mode="list",
             ragged=False, out="bfloat16"),
        # eight sequences of 96k, 4096 selected tokens for each KV head
        dict(name="attn_96k_b8", op="attn", batch=8, kv=8, g=4, d=128, ctx=98304, bs=32, kb=256, kt=4096, mode="list",
             ragged=False, out="float32"),
        # the same heads over a slot cache of 2 K_b blocks (offloaded KV), an odd number of tokens
        dict(name="attn_paged_96k", op="attn", batch=3, kv=8, g=4, d=128, ctx=98304, bs=32, kb=192, kt=2047,
             mode="paged", ragged=True, out="bfloat16"),
        # every token of eight sequences: the largest call
        dict(name="attn_dense_96k_b8", op="attn", batch=8, kv=8, g=4, d=128, ctx=98304, bs=32, kb=256, kt=4096,
             mode="dense", ragged=False, out="bfloat16"),
        # weights of the 96k step's 4096 tokens, bf16 keys
        dict(name="weights_96k_b8", op="weights", batch=8, kv=8, g=4, d=128, ctx=98304, bs=32, kb=256, kt=4096,
             keys="bf16", mode="list", ragged=False),
        # 64 heads on one shared latent of 576 channels
        dict(name="weights_latent_64k_b4", op="weights", batch=4, kv=1, g=64, d=576, ctx=65536, bs=64, kb=128, kt=2048,
             keys="latent", mode="list", ragged=False),
        # fp32 keys, ragged short sequences, every token
        dict(name="weights_f32_ragged", op="weights", batch=3, kv=2, g=2, d=64, ctx=1999, bs=32, kb=16, kt=256,
             keys="f32", mode="dense", ragged=True),
        # half of a 96k cache evicted: K and V rows in bf16
        dict(name="evict_96k_b8", op="evict", batch=8, kv=8, d=128, ctx=98304, budget=49152, sink=4, recent=512,
             store="bf16", ragged=False),
        # a 4-bit cache of one sequence, a sixth of it evicted
        dict(name="evict_kv4_48k", op="evict", batch=1, kv=8, d=128, ctx=49152, budget=40960, sink=4, recent=256,
             store="kv4", ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "weights", "evict"])
    batch, kv, d = _log(rng, 1, 8), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128])
    bs, ragged = rng.choice([16, 32, 64]), rng.random() < 0.5
    ctx = _log(rng, 256, 98304)
    if op == "store":
        rows = rng.choice([1, 1, _log(rng, 1, ctx)])
        return dict(op=op, batch=_log(rng, 1, 64) if rows == 1 else min(batch, 4), kv=kv, d=d,
                    ctx=min(ctx, 16384) if rows == 1 else ctx, rows=rows,
                    old=rng.randrange(0, (min(ctx, 16384) if rows == 1 else ctx) - rows + 1), bs=bs,
                    r=rng.choice([8, 16, 32]))
    if op == "evict":
        recent, sink = rng.choice([1, 17, 128]), rng.choice([0, 4, 5])
        return dict(op=op, batch=batch, kv=kv, d=d, ctx=ctx, budget=max(recent + sink, int(ctx * rng.uniform(0.2, 0.95))),
                    sink=sink, recent=recent, store=rng.choice(["bf16", "kv4"]), ragged=ragged)
    kt = _log(rng, 1, 4096)
    kb = max(1, min(1024, 16384 // bs, -(-ctx // bs), _log(rng, max(1, -(-kt // bs)), 256)))
    case = dict(op=op, batch=batch, kv=kv, g=rng.choice([1, 2, 4, 8, 16]), d=d, ctx=ctx, bs=bs, kb=kb, kt=kt,
                mode=rng.choice(["list", "list", "dense"]), ragged=ragged)
    if op == "attn":
        case = dict(case, mode=rng.choice(["list", "paged", "dense"]), out=rng.choice(["bfloat16", "float32"]))
    else:
        case["keys"] = rng.choice(["bf16", "bf16", "f32", "kv4", "latent"])
        if case["keys"] == "latent":
            case.update(kv=1, d=576, g=rng.choice([16, 32, 64]), batch=min(batch, 4))
    if case["mode"] == "dense":  # no more than the largest listed case
        case["ctx"] = min(ctx, 64 * 98304 * 4 // (case["batch"] * case["kv"] * max(4, case["g"])))
    return case


# ------------------------------------------------------------------------------- 4-bit values, plain form
def _scale_of(b):
    """Scale bytes -> fp32: the fp16 number with the bits b << 7."""
    return (b.to(torch.int16) << 7).view(torch.float16).to(F32)


def _encode(x):
    """Rows [..., d] -> (codes uint8 [..., d / 2], scale bytes uint8 [..., d / 16]), decided in fp32."""
    g = x.to(F32).unflatten(-1, (-1, 16))
    amax = g.abs().amax(-1)
    s = amax / 6.0
    bits = s.view(torch.int32)
    normal = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (112 << 3)
    b = torch.where(s < 2.0 ** -14, (s * 2.0 ** 17).round().to(torch.int32), normal).clamp(max=0xE2)
    fine = amax.isfinite()
    b = torch.where(fine, b, torch.full_like(b, 0xFF)).to(torch.uint8)
    keep = (fine & (b > 0))[..., None]
    y = torch.where(keep, g / _scale_of(torch.where(keep[..., 0], b, torch.full_like(b, 0x78)))[..., None], torch.zeros_like(g))
    a = y.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    c = (m | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), b


def _decode(codes, scales):
    """(codes, scale bytes) -> fp32 rows [..., d]: an e2m1 code's bits are those of an fp16 number times 2^-14."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int16)
    v = (((n & 8) << 12) | ((n & 7) << 9)).view(torch.float16).to(F32) * 2.0 ** 14
    return (v.unflatten(-1, (-1, 16)) * _scale_of(scales)[..., None]).flatten(-2)


def _records(K, V):
    """K and V rows -> records uint8 [..., 9 d / 8]."""
    kc, ks = _encode(K)
    vc, vs = _encode(V)
    return torch.cat((kc, ks, vs, vc), -1)


def _k_of(rec, d):
    return _decode(rec[..., :d // 2], rec[..., d // 2:d // 2 + d // 16])


def _v_of(rec, d):
    return _decode(rec[..., d // 2 + d // 8:], rec[..., d // 2 + d // 16:d // 2 + d // 8])


# ----------------------------------------------------------------------------------------------- inputs
def _lens(case, gen):
    B, ctx = case["batch"], case["ctx"]
    if not case["ragged"]:
        return torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    return torch.randint(1, ctx + 1, (B,), generator=gen, device="cuda").to(torch.int32)


def _rows(gen, shape, dtype, outliers=True):
    """N(0, 1) rows, a fixed set of channels scaled by 5 (keys have such channels)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    if outliers:
        x[..., 3::shape[-1] // 8] *= 5
    return x


def _selection(case, lens, gen):
    """Ascending distinct tokens of k_b blocks of each (sequence, KV head), -1 padded, and the blocks."""
    B, H, bs, kt = case["batch"], case["kv"], case["bs"], case["kt"]
    nb = -(-case["ctx"] // bs)
    kb = min(case["kb"], nb)
    score = torch.rand((B, H, nb), generator=gen, device="cuda")
    score = torch.where(torch.arange(nb, device="cuda") * bs < lens[:, None, None], score, score - 2)
    top = score.topk(kb, -1)
    blocks = torch.where(top.values >= 0, top.indices, -1)
    cand = blocks[..., None] * bs + torch.arange(bs, device="cuda")
    cand = torch.where((blocks[..., None] >= 0) & (cand < lens[:, None, None, None]), cand, -1).flatten(2)
    pick = torch.where(cand >= 0, torch.rand(cand.shape, generator=gen, device="cuda"), torch.full(cand.shape, -1.0, device="cuda"))
    top = pick.topk(min(kt, cand.shape[-1]), -1)
    big = case["ctx"] + 1
    tok = torch.where(top.values >= 0, cand.gather(2, top.indices), big).sort(-1).values
    tok = torch.where(tok == big, -1, tok)
    if tok.shape[-1] < kt:
        tok = torch.cat((tok, torch.full((B, H, kt - tok.shape[-1]), -1, device="cuda", dtype=tok.dtype)), -1)
    return tok.to(torch.int32).contiguous(), blocks.to(torch.int32)


def _shape(case, dtype=1, out=0):
    from two_level_sparse_quest_b200 import tls as T

    latent = case.get("keys") == "latent"
    bs = case.get("bs", 64)
    return T.make_shape(batch=case["batch"], n_q_heads=case["kv"] * case.get("g", 4), n_kv_heads=case["kv"],
                        d_qk=case["d"], d_v=512 if latent else case["d"], block_size=bs, n_label=case.get("r", 16),
                        k_b=case.get("kb", 1), k_t=case.get("kt", 1), max_ctx=case["ctx"], kv_dtype=dtype,
                        out_dtype=out, v_is_k_prefix=latent)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    B, H, d, ctx, op = case["batch"], case["kv"], case["d"], case["ctx"], case["op"]
    if op == "store":
        n, nb = case["rows"], -(-ctx // case["bs"])
        st["K"], st["V"] = _rows(gen, (B, H, n, d), BF16), _rows(gen, (B, H, n, d), BF16, False)
        st["old"] = torch.full((B,), case["old"], dtype=torch.int32, device="cuda")
        st["new"] = st["old"] + n
        st["label"] = torch.randperm(d, generator=gen, device="cuda")[:case["r"]].sort().values.to(torch.int32)
        st["cache"] = torch.zeros((B, H, ctx, 9 * d // 8), dtype=torch.uint8, device="cuda")
        lo = -_rows(gen, (B, H, nb, 1, d), BF16).abs()  # the summary that the old tokens left
        st["meta"] = torch.cat((-lo, lo), 3)
        st["slab"] = torch.zeros((B, H, ctx, case["r"]), dtype=BF16, device="cuda")
        st["Kb"], st["Vb"] = torch.empty_like(st["K"]), torch.empty_like(st["V"])
        return st
    lens = st["lens"] = _lens(case, gen)
    if op == "evict":
        w = torch.exp(2 * torch.randn((B, H, ctx), generator=gen, device="cuda")) * 1e-3
        st["weights"] = torch.where(torch.rand((B, H, ctx), generator=gen, device="cuda") < 0.4, 0.0, w)
        st["w"] = torch.empty_like(st["weights"])
        st["keep"] = torch.empty((B, H, case["budget"]), dtype=torch.int32, device="cuda")
        st["new"] = torch.empty_like(lens)
        if case["store"] == "kv4":
            st["rows"] = [torch.randint(0, 256, (B, H, ctx, 9 * d // 8), generator=gen, device="cuda", dtype=torch.uint8)]
        else:
            st["rows"] = [_rows(gen, (B, H, ctx, d), BF16, False) for _ in range(2)]
        return st
    G, keys = case["g"], case.get("keys", "kv4")
    ktype = F32 if keys == "f32" else BF16
    st["q"] = _rows(gen, (B, H * G, d), ktype, False)
    n, per = ctx, None
    if case["mode"] == "dense":
        st["tok"] = None
    else:
        st["tok"], blocks = _selection(case, lens, gen)
    if case["mode"] == "paged":  # 2 K_b slots; the selected blocks lie in some of them, in any order
        nb = -(-ctx // case["bs"])
        slots = 2 * min(case["kb"], nb)
        n = slots * case["bs"]
        perm = torch.rand((B, H, slots), generator=gen, device="cuda").argsort(-1)[..., :blocks.shape[-1]].to(torch.int32)
        table = torch.full((B, H, nb + 1), -1, dtype=torch.int32, device="cuda")
        table.scatter_(2, torch.where(blocks >= 0, blocks, nb).long(), perm)
        st["table"], st["slots"] = table[..., :nb].contiguous(), slots
    if keys == "kv4":
        cache = torch.empty((B, H, n, 9 * d // 8), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // max(1, n * d * H))
        for b in range(0, B, step):
            shape = (min(step, B - b), H, n, d)
            cache[b:b + step] = _records(_rows(gen, shape, BF16), _rows(gen, shape, BF16, False))
        st["cache"] = cache
    else:
        st["K"] = _rows(gen, (B, H, n, d), ktype)
    if op == "weights":
        st["weights"] = 0.01 * torch.rand((B, H, ctx), generator=gen, device="cuda")
        # the log-sum-exp that the step's attention returned
        s = _logits(st, F32)
        st["lse"] = torch.logsumexp(s, -1).flatten(1).contiguous()
        return st
    st["out"] = torch.empty((B, H * G, d), dtype=getattr(torch, case["out"]), device="cuda")
    st["lse"] = torch.empty((B, H * G), dtype=F32, device="cuda")
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _place(st):
    """(index of each token's row in the cache, whether the token takes part), [B, H, n]."""
    case = st["case"]
    B, H = case["batch"], case["kv"]
    if st["tok"] is None:
        t = torch.arange(case["ctx"], device="cuda")
        return None, (t < st["lens"][:, None, None]).expand(B, H, -1)
    tok = st["tok"].long()
    if case["mode"] != "paged":
        return tok.clamp(min=0), tok >= 0
    slot = st["table"].gather(2, tok.clamp(min=0) // case["bs"]).long()
    ok = (tok >= 0) & (slot >= 0)
    return torch.where(ok, slot * case["bs"] + tok % case["bs"], 0), ok


def _take(x, at):
    return x if at is None else x.gather(2, at[..., None].expand(-1, -1, -1, x.shape[-1]))


def _logits(st, dtype):
    """tau q . k of every token and head [B, H, G, n], -inf where the token takes no part."""
    case = st["case"]
    at, ok = _place(st)
    d = case["d"]
    K = _take(st["K"], at).to(dtype) if "K" in st else _k_of(_take(st["cache"], at), d).to(dtype)
    q = st["q"].to(dtype).unflatten(1, (case["kv"], case["g"]))
    return ((q @ K.mT) * (1 / math.sqrt(d))).masked_fill(~ok[:, :, None], -math.inf)


def run(st):
    case = st["case"]
    if own:
        return _own(st)
    op, d = case["op"], case["d"]
    if op == "store":
        return _plain_store(st)
    if op == "evict":
        return _plain_evict(st)
    s = _logits(st, F32)
    if op == "attn":
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
        z = p.sum(-1, keepdim=True)
        at, ok = _place(st)
        V = _v_of(_take(st["cache"], at), d)
        o = torch.where(z > 0, (p @ V) / z, 0.0)
        return {"out": o.flatten(1, 2).to(st["out"].dtype), "lse": (m + torch.log(z)).flatten(1)}
    lse = st["lse"].unflatten(1, (case["kv"], case["g"]))[..., None]
    w = torch.where(lse == -math.inf, 0.0, torch.exp(s - lse)).sum(2)
    at, ok = _place(st)
    if at is None:
        st["weights"] += w
    else:
        st["weights"].scatter_add_(2, at, torch.where(ok, w, 0.0))
    return {"weights": st["weights"]}


def _plain_store(st):
    case = st["case"]
    d, bs, old, n = case["d"], case["bs"], case["old"], case["rows"]
    st["cache"][:, :, old:old + n] = _records(st["K"], st["V"])
    st["slab"][:, :, old:old + n] = st["K"][..., st["label"].long()]
    # rows by block: [first block, last block] of the appended range, with -inf / inf around it
    b0, b1 = old // bs, (old + n - 1) // bs + 1
    pad = (old - b0 * bs, b1 * bs - old - n)
    by = lambda v: torch.nn.functional.pad(st["K"], (0, 0) + pad, value=v).unflatten(2, (-1, bs))
    new = torch.stack((by(-math.inf).amax(3), by(math.inf).amin(3)), 3)
    had = st["meta"][:, :, b0:b1]
    if pad[0]:  # the first block had rows already
        new[:, :, 0, 0] = torch.maximum(new[:, :, 0, 0], had[:, :, 0, 0])
        new[:, :, 0, 1] = torch.minimum(new[:, :, 0, 1], had[:, :, 0, 1])
    st["meta"][:, :, b0:b1] = new
    rec = st["cache"][:, :, old:old + n]
    return {"K": _k_of(rec, d).to(BF16), "V": _v_of(rec, d).to(BF16), "meta": st["meta"], "slab": st["slab"]}


def _plain_evict(st):
    case = st["case"]
    ctx, budget = case["ctx"], case["budget"]
    w = st["w"]
    w.copy_(st["weights"])
    t = torch.arange(ctx, device="cuda")
    lens = st["lens"][:, None, None]
    rank = torch.where((t < case["sink"]) | (t >= lens - case["recent"]), math.inf, w)
    rank = torch.where(t < lens, rank, -math.inf)
    order = rank.sort(stable=True, dim=-1, descending=True).indices[..., :budget]
    new = st["lens"].clamp(max=budget)
    live = torch.arange(budget, device="cuda") < new[:, None, None]
    keep = torch.where(live, order, ctx).sort(-1).values
    at = keep.clamp(max=ctx - 1)
    rows = st["rows"] + [w[..., None]]
    for x in rows:
        x[:, :, :budget] = torch.where(live[..., None], _take(x, at), x[:, :, :budget])
    w.masked_fill_((t >= new[:, None, None]) & (t < lens), 0.0)
    return {"keep": torch.where(live, keep, -1).to(torch.int32), "new": new, "rows": st["rows"], "weights": w}


# ---------------------------------------------------------------------------------- the library's calls
def _own(st):
    from two_level_sparse_quest_b200 import tls as T

    case, op = st["case"], st["case"]["op"]
    if "shape" not in st:
        st["shape"] = _shape(case, 0 if case.get("keys") == "f32" else 1, 0 if case.get("out") == "float32" else 1)
    s = st["shape"]
    if op == "store":
        T.tls_kv4_append(s, st["K"], st["V"], st["old"], st["new"], case["rows"], st["cache"], st["label"], st["meta"], st["slab"])
        T.tls_kv4_read(s, st["cache"], st["old"], st["new"], case["rows"], st["Kb"], st["Vb"])
        return {"K": st["Kb"], "V": st["Vb"], "meta": st["meta"], "slab": st["slab"]}
    if op == "evict":
        st["w"].copy_(st["weights"])
        T.tls_evict_select(s, case["budget"], case["sink"], case["recent"], st["w"], st["lens"], st["keep"], st["new"])
        T.tls_evict_compact(s, case["budget"], st["keep"], st["lens"], st["rows"], st["w"])
        return {"keep": st["keep"], "new": st["new"], "rows": st["rows"], "weights": st["w"]}
    if op == "attn":
        if "ws" not in st:
            st["ws"] = torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda")
        T.tls_kv4_attn_decode(s, st["q"], st["cache"], st["out"], st["lse"], token_idx=st["tok"],
                              seq_lens=st["lens"] if st["tok"] is None else None, slot_of_block=st.get("table"),
                              n_slots=st.get("slots", 0), ws=st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    call = T.tls_kv4_accum_weights if case["keys"] == "kv4" else T.tls_accum_weights
    call(s, st["q"], st["cache"] if case["keys"] == "kv4" else st["K"], st["lse"], st["weights"],
         token_idx=st["tok"], seq_lens=st["lens"] if st["tok"] is None else None)
    return {"weights": st["weights"]}


# ------------------------------------------------------------------------------------------ work, exact
def _tokens(case):
    """Tokens that take part, over all (sequence, KV head) pairs; ragged lengths are half the capacity on average."""
    full = case["batch"] * case["kv"]
    mean = (case["ctx"] + 1) / 2 if case["ragged"] else case["ctx"]
    return full * (mean if case.get("mode") == "dense" or case["op"] == "evict" else min(case["kt"], mean))


def work(case):
    B, H, d, op = case["batch"], case["kv"], case["d"], case["op"]
    if op == "store":
        rows = B * H * case["rows"]
        blocks = B * H * (case["rows"] / case["bs"] + 1)
        # rows in, records out, label rows out, the touched summaries out, the rows read back
        return {"bytes": rows * (4 * d + 9 * d / 8 + 2 * case["r"] + 4 * d) + blocks * 4 * d, "flops": 8.0 * rows * d}
    if op == "evict":
        n = _tokens(case)
        kept = min(n, B * H * case["budget"])
        row = 9 * d / 8 if case["store"] == "kv4" else 4 * d
        return {"bytes": 4 * n + 4 * kept + 2 * kept * (row + 4), "flops": n}
    n, G = _tokens(case), case["g"]
    ids = 0 if case["mode"] == "dense" else 4 * n
    io = B * H * G * (2 * d + 4)
    if op == "attn":
        out = B * H * G * d * (4 if case["out"] == "float32" else 2)
        return {"bytes": n * 9 * d / 8 + ids + io + out, "flops": 4.0 * n * G * d}
    row = {"bf16": 2 * d, "latent": 2 * d, "f32": 4 * d, "kv4": 9 * d / 16}[case["keys"]]
    return {"bytes": n * (row + 8) + ids + io, "flops": 2.0 * n * G * d}


def _scales64():
    """The 226 finite scales up to 10240 in 64 bits, from their definition."""
    b = torch.arange(0xE3, device="cuda")
    e, m = (b >> 3).double(), (b & 7).double()
    return torch.where(e == 0, m * 2.0 ** -17, (1 + m / 8) * torch.exp2(e - 15))


def _nearest(x, table):
    """Index of the nearest of `table` (ascending), the even index where two are as near."""
    lo = (torch.searchsorted(table, x, right=True) - 1).clamp(0, len(table) - 2)
    below, above = x - table[lo], table[lo + 1] - x
    return lo + ((above < below) | ((above == below) & (lo % 2 == 1))).long()


def _exact_store(st):
    case = st["case"]
    grid, scales = torch.tensor(E2M1, dtype=torch.float64, device="cuda"), _scales64()

    def stored(x):
        x = x.double().unflatten(-1, (-1, 16))
        s = scales[_nearest(x.abs().amax(-1) / 6, scales)][..., None]
        y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
        return (grid[_nearest(y, grid)] * torch.sign(x) * s).flatten(-2)

    old, n, bs = case["old"], case["rows"], case["bs"]
    meta, slab = st["meta"].double(), st["slab"].double()
    for i, c in enumerate(st["label"].tolist()):
        slab[:, :, old:old + n, i] = st["K"][..., c].double()
    for j in range(old // bs, (old + n - 1) // bs + 1):
        x = st["K"][:, :, max(0, j * bs - old):(j + 1) * bs - old].double()
        hi, lo = x.amax(2), x.amin(2)
        if j * bs < old:
            hi, lo = torch.maximum(hi, meta[:, :, j, 0]), torch.minimum(lo, meta[:, :, j, 1])
        meta[:, :, j, 0], meta[:, :, j, 1] = hi, lo
    return {"K": stored(st["K"]), "V": stored(st["V"]), "meta": meta, "slab": slab}


def _exact_evict(st):
    case = st["case"]
    B, H, budget = case["batch"], case["kv"], case["budget"]
    rows, w = [x.clone() for x in st["rows"]], st["weights"].double()
    for b in range(B):
        n = int(st["lens"][b])
        if n <= budget:
            continue
        for h in range(H):
            mid = st["weights"][b, h, case["sink"]:n - case["recent"]].cpu().numpy()
            best = (-mid).argsort(kind="stable")[:budget - case["sink"] - case["recent"]] + case["sink"]
            keep = torch.tensor(sorted(list(range(case["sink"])) + best.tolist() + list(range(n - case["recent"], n))), device="cuda")
            for x, y in zip(rows, st["rows"]):
                x[b, h, :budget] = y[b, h][keep]
            w[b, h, :n] = 0
            w[b, h, :budget] = st["weights"][b, h][keep].double()
    return {"keep": None, "new": None, "rows": rows, "weights": w}


def exact(case, seed):
    """In 64 bits, from the definitions, one (sequence, KV head) at a time; whole numbers have no such value."""
    st = prepare(case, seed)
    if case["op"] in ("store", "evict"):
        return _exact_store(st) if case["op"] == "store" else _exact_evict(st)
    B, H, G, d, bs = case["batch"], case["kv"], case["g"], case["d"], case.get("bs")
    f64 = torch.float64
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=f64, device="cuda")
    scale = _scales64()

    def half(rec, c0, s0):
        c = rec[:, c0:c0 + d // 2].long()
        v = torch.empty((len(rec), d), dtype=f64, device="cuda")
        v[:, 0::2], v[:, 1::2] = table[c & 15], table[c >> 4]
        return v * scale[rec[:, s0:s0 + d // 16].long()].repeat_interleave(16, 1)

    outs, lses = [], []
    acc = st["weights"].double() if case["op"] == "weights" else None
    for b in range(B):
        for h in range(H):
            if st["tok"] is None:
                tok = torch.arange(int(st["lens"][b]), device="cuda")
            else:
                tok = st["tok"][b, h].long()
                tok = tok[tok >= 0]
            at = tok
            if case["mode"] == "paged":
                slot = st["table"][b, h][tok // bs].long()
                tok, slot = tok[slot >= 0], slot[slot >= 0]
                at = slot * bs + tok % bs
            rec = st["cache"][b, h][at] if "cache" in st else None
            K = st["K"][b, h][at].double() if rec is None else half(rec, 0, d // 2)
            a = st["q"][b, h * G:(h + 1) * G].double() @ K.T / math.sqrt(d)
            if acc is not None:
                lse = st["lse"][b, h * G:(h + 1) * G].double()
                if len(tok):
                    acc[b, h].index_add_(0, tok, torch.exp(a - lse[:, None]).sum(0))
                continue
            lses.append(torch.logsumexp(a, -1) if len(tok) else torch.full((G,), -math.inf, dtype=f64, device="cuda"))
            outs.append(torch.softmax(a, -1) @ half(rec, d // 2 + d // 8, d // 2 + d // 16) if len(tok)
                        else torch.zeros((G, d), dtype=f64, device="cuda"))
    if acc is not None:
        return {"weights": acc}
    return {"out": torch.cat(outs).view(B, H * G, d), "lse": torch.cat(lses).view(B, H * G)}
