"""Accumulated attention weight and the eviction by it, on the GPU, against the 64-bit forms in tests/_kv4.py:
sums within their derived bounds, kept ids and moved rows exactly; and a decode loop over a 4-bit cache that uses
the operators together."""
import numpy as np
import pytest
import torch

from tests import _kv4 as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from two_level_sparse_quest_b200 import build

    build.build()
    from two_level_sparse_quest_b200 import tls

    tls.tls_device_error(clear=True)
    return tls


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make(T, B, H, G, d, ctx, kt=1, dtype=1, bs=32):
    latent = d == 576
    return T.make_shape(batch=B, n_q_heads=H * G, n_kv_heads=H, d_qk=d, d_v=512 if latent else d, block_size=bs,
                        n_label=16, k_b=1, k_t=kt, max_ctx=ctx, kv_dtype=dtype, v_is_k_prefix=latent)


# ----------------------------------------------------------------------------------------------- weights
def check_weights(T, B, H, G, d, ctx, kind, tokens=None, lens=None, seed=3):
    rng = np.random.default_rng(seed)
    kt = len(tokens[0][0]) if tokens else 1
    s = make(T, B, H, G, d, ctx, kt, 0 if kind == "f32" else 1)
    ktype = torch.float32 if kind == "f32" else BF16
    q = torch.from_numpy(rng.standard_normal((B, H * G, d)).astype(np.float32)).to(ktype)
    x = rng.standard_normal((B, H, ctx, d)).astype(np.float32)
    x[..., 3::d // 8] *= 5
    K = torch.from_numpy(x).to(ktype)
    if kind == "kv4":
        keys = torch.from_numpy(R.records(f64(K), f64(K))).cuda()
        K64 = R.split(keys.cpu().numpy(), d)[0]
    else:
        keys, K64 = K.cuda(), f64(K)
    tau = 1 / np.sqrt(d)
    ids = tokens if tokens else [[list(range(n))] * H for n in lens]
    lse = np.full((B, H * G), -np.inf, np.float32)
    for b in range(B):
        for h in range(H):
            t = [j for j in ids[b][h] if 0 <= j < ctx]
            if t:
                lse[b, h * G:(h + 1) * G] = R.attention(f64(q[b, h * G:(h + 1) * G]), K64[b, h], K64[b, h], t, tau)[1]
    acc0 = rng.random((B, H, ctx)).astype(np.float32) * 0.01
    kw = dict(token_idx=i32(tokens)) if tokens else dict(seq_lens=i32(lens))
    call = T.tls_kv4_accum_weights if kind == "kv4" else T.tls_accum_weights
    got = []
    for _ in range(2):
        w = torch.from_numpy(acc0).cuda()
        call(s, q.cuda(), keys, torch.from_numpy(lse).cuda(), w, **kw)
        got.append(w.cpu())
    assert torch.equal(got[0], got[1])  # the same bits
    for b in range(B):
        for h in range(H):
            t = [j for j in ids[b][h] if 0 <= j < ctx]
            add, tol = R.weights(f64(q[b, h * G:(h + 1) * G]), K64[b, h], lse[b, h * G:(h + 1) * G], t, tau, ctx)
            want = acc0[b, h].astype(np.float64) + add
            many = max(1, max((ids[b][h].count(j) for j in set(t)), default=1)) if tokens else 1
            err = np.abs(f64(got[0][b, h]) - want)
            assert (err <= tol + many * R.U32 * want).all(), (b, h, float((err - tol).max()))
            assert (err[add == 0] == 0).all()


def lists(rng, B, H, ctx, kt, pad=0):
    t = np.full((B, H, kt), -1, np.int64)
    for b in range(B):
        for h in range(H):
            n = min(kt - pad, ctx)
            t[b, h, :n] = rng.permutation(ctx)[:n]
    return t.tolist()


@pytest.mark.parametrize("kind,d,G", [("bf16", 64, 1), ("bf16", 128, 4), ("bf16", 128, 16), ("bf16", 64, 32), ("bf16", 128, 64),
                                      ("f32", 64, 2), ("f32", 128, 8), ("f32", 64, 64), ("kv4", 64, 4), ("kv4", 128, 1),
                                      ("kv4", 128, 16), ("kv4", 64, 32), ("kv4", 128, 64), ("latent", 576, 4),
                                      ("latent", 576, 12), ("latent", 576, 64), ("latent", 576, 128)])
def test_weights_types_and_heads(T, kind, d, G):
    rng = np.random.default_rng(G)
    B, H = 2, 1 if d == 576 or G > 8 else 3
    check_weights(T, B, H, G, d, 333, kind, tokens=lists(rng, B, H, 333, 75, pad=2))
    check_weights(T, B, H, G, d, 201, kind, lens=[201, 0])


@pytest.mark.parametrize("kind", ["bf16", "f32", "kv4"])
@pytest.mark.parametrize("n", [1, 7, 8, 15, 16, 17, 127, 128, 129, 1000])
def test_weights_lengths(T, kind, n):
    rng = np.random.default_rng(n)
    check_weights(T, 1, 2, 4, 128, 1001, kind, tokens=lists(rng, 1, 2, 1001, n))
    check_weights(T, 3, 1, 4, 64, 1001, kind, lens=[n, 1, 1001])


@pytest.mark.parametrize("kind", ["bf16", "f32", "kv4"])
def test_weights_masked_and_repeated_ids(T, kind):
    bad = [-1, 5, -9, 99, 5, 100, 2 ** 31 - 1, 0, 5] + [-1] * 30 + [98]
    check_weights(T, 1, 3, 4, 64, 100, kind, tokens=[[bad, [-1] * len(bad), [100] * len(bad)]])


def test_weights_of_heads_without_tokens_and_with_nan(T):
    """lse = -inf adds nothing even where keys are NaN-free but listed; a NaN key reaches its own token only."""
    s = make(T, 1, 1, 4, 128, 64, 3)
    q = torch.randn((1, 4, 128), device="cuda").to(BF16)
    K = torch.randn((1, 1, 64, 128), device="cuda").to(BF16)
    w = torch.zeros((1, 1, 64), device="cuda")
    T.tls_accum_weights(s, q, K, torch.full((1, 4), -float("inf"), device="cuda"), w, token_idx=i32([[[1, 2, 3]]]))
    assert (w == 0).all()
    K[0, 0, 2, 7] = float("nan")
    K[0, 0, 9] = float("inf")
    T.tls_accum_weights(s, q, K, torch.zeros((1, 4), device="cuda"), w, token_idx=i32([[[1, 2, 3]]]))
    assert w[0, 0, 2].isnan() and w[0, 0, [0, 1, 3, 9]].isfinite().all() and w[0, 0, 1] > 0 and w[0, 0, 0] == 0


# -------------------------------------------------------------------------------------------------- select
def check_select(T, w, lens, budget, n_sink, n_recent, H=None):
    B, H, ctx = w.shape
    s = make(T, B, H, 1, 64, ctx, bs=max(1, -(-ctx // 16384)))
    keep = torch.full((B, H, budget), -7, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    T.tls_evict_select(s, budget, n_sink, n_recent, torch.from_numpy(w).cuda(), i32(lens), keep, new)
    torch.cuda.synchronize()
    got = keep.cpu().numpy()
    assert new.tolist() == [min(max(n, 0), budget, ctx) for n in lens]
    for b in range(B):
        for h in range(H):
            want = R.keep(w[b, h], min(max(lens[b], 0), ctx), budget, n_sink, n_recent)
            np.testing.assert_array_equal(got[b, h, :len(want)], want)
            assert (got[b, h, len(want):] == -1).all()


def heavy(rng, shape, zeros=0.4):
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32) * np.float32(1e-3)
    return np.where(rng.random(shape) < zeros, np.float32(0), w).astype(np.float32)


@pytest.mark.parametrize("ctx", [1, 2, 31, 33, 100, 511, 512, 513, 4095, 4097, 8193, 20000, 40001])
def test_select_lengths(T, ctx):
    rng = np.random.default_rng(ctx)
    for budget in sorted({1, max(1, ctx // 3), ctx - 1 or 1, ctx}):
        sink, recent = min(4, budget // 2), min(17, budget - budget // 2)
        check_select(T, heavy(rng, (3, 2, ctx)), [ctx, ctx // 2, 1], budget, sink, recent)


def test_select_ragged_empty_and_clamped_lengths(T):
    rng = np.random.default_rng(4)
    check_select(T, heavy(rng, (6, 2, 900)), [0, 1, 300, 301, 900, 5000], 300, 2, 100)
    check_select(T, heavy(rng, (2, 1, 900)), [-5, 900], 7, 0, 0)
    check_select(T, heavy(rng, (1, 1, 900)), [900], 40, 10, 30)  # nothing but the protected ones


@pytest.mark.parametrize("ctx", [3000, 9000])
def test_select_ties_and_special_weights(T, ctx):
    rng = np.random.default_rng(6)
    for w in (np.zeros((1, 2, ctx)), np.full((1, 2, ctx), 0.25), np.where(rng.random((1, 2, ctx)) < 0.5, 0.0, -0.0),
              rng.integers(0, 3, (1, 2, ctx)) * 0.5, -rng.random((1, 2, ctx)), rng.integers(-2, 2, (1, 2, ctx)),
              np.where(rng.random((1, 2, ctx)) < 0.2, np.nan, rng.random((1, 2, ctx))),
              np.where(rng.random((1, 2, ctx)) < 0.3, np.inf, rng.random((1, 2, ctx))),
              np.full((1, 2, ctx), np.nan), np.full((1, 2, ctx), -np.inf), np.full((1, 2, ctx), np.inf),
              np.float32(1) + rng.integers(0, 9, (1, 2, ctx)) * np.float32(2.0 ** -23),
              rng.random((1, 2, ctx)) * 1e-42):
        for budget in (1, 1000, ctx - 1):
            check_select(T, w.astype(np.float32), [ctx], budget, min(3, budget // 2), min(64, budget // 2))


def test_select_beyond_shared_memory(T):
    """A slice of more keys than a CTA holds on chip: the rest is read again."""
    rng = np.random.default_rng(8)
    w = heavy(rng, (1, 1, 500000))
    check_select(T, w, [500000], 200000, 4, 512)
    check_select(T, w, [499999], 400001, 0, 1)


# ------------------------------------------------------------------------------------------------- compact
def run_compact(T, B, H, ctx, lens, budget, keeps, row_bytes, with_weights=True, offset=0, seed=1):
    rng = np.random.default_rng(seed)
    s = make(T, B, H, 1, 64, ctx, bs=max(1, -(-ctx // 16384)))
    arrays, base = [], []
    for rb in row_bytes:
        a = rng.integers(0, 256, (B, H, ctx, rb), dtype=np.uint8)
        store = torch.zeros(a.size + 64, dtype=torch.uint8, device="cuda")
        store[offset:offset + a.size] = torch.from_numpy(a.reshape(-1)).cuda()
        arrays.append((a, store))
        base.append((store.data_ptr() + offset, rb))
    w0 = rng.random((B, H, ctx)).astype(np.float32) + 1
    w = torch.from_numpy(w0).cuda()
    keep = np.full((B, H, budget), -1, np.int32)
    for b in range(B):
        for h in range(H):
            keep[b, h, :len(keeps[b][h])] = keeps[b][h]
    T.tls_evict_compact(s, budget, torch.from_numpy(keep).cuda(), i32(lens), base, w if with_weights else None)
    torch.cuda.synchronize()
    gw = w.cpu().numpy()
    for (a, store), rb in zip(arrays, row_bytes):
        got = store.cpu().numpy()
        assert (got[:offset] == 0).all() and (got[offset + a.size:] == 0).all()
        got = got[offset:offset + a.size].reshape(a.shape)
        for b in range(B):
            for h in range(H):
                k = keeps[b][h]
                np.testing.assert_array_equal(got[b, h, :len(k)], a[b, h, k])
                np.testing.assert_array_equal(got[b, h, len(k):], a[b, h, len(k):])  # left as they were
    for b in range(B):
        for h in range(H):
            k, n = keeps[b][h], lens[b]
            want = w0[b, h].copy()
            if with_weights:
                want[:n] = 0
                want[:len(k)] = w0[b, h, k]
            np.testing.assert_array_equal(gw[b, h], want)


def random_keeps(rng, B, H, lens, budget):
    return [[np.sort(rng.permutation(n)[:min(n, budget)]) if n > budget else np.arange(n) for _ in range(H)] for n in lens]


@pytest.mark.parametrize("rb", [1, 2, 3, 4, 6, 8, 12, 16, 32, 72, 144, 256, 1152, 13316])
def test_compact_row_sizes(T, rb):
    rng = np.random.default_rng(rb)
    ctx = 700 if rb < 4096 else 90
    lens = [ctx, ctx // 2, 0, 1]
    run_compact(T, 4, 2, ctx, lens, ctx // 3, random_keeps(rng, 4, 2, lens, ctx // 3), [rb])


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
def test_compact_several_arrays_and_alignments(T, offset):
    rng = np.random.default_rng(offset)
    lens = [501, 333]
    run_compact(T, 2, 3, 501, lens, 260, random_keeps(rng, 2, 3, lens, 260), [256, 256, 32, 72], offset=offset)
    run_compact(T, 2, 3, 501, lens, 260, random_keeps(rng, 2, 3, lens, 260), [144], with_weights=False, offset=offset)


def test_compact_long_and_few_groups(T):
    """Many chunks, each overwriting rows that others still read a moment before; one row evicted, and nearly all."""
    n = 30000
    for seed in range(3):
        rng = np.random.default_rng(seed)
        run_compact(T, 1, 1, n, [n], n - 1, [[np.delete(np.arange(n), rng.integers(0, n))]], [144, 16], seed=seed)
        run_compact(T, 1, 2, n, [n], 20000, random_keeps(rng, 1, 2, [n], 20000), [256, 256], seed=seed)
        run_compact(T, 1, 1, n, [n], 40, random_keeps(rng, 1, 1, [n], 40), [72], seed=seed)


def test_compact_caller_list_shorter_than_the_budget(T):
    run_compact(T, 1, 2, 100, [90], 50, [[np.array([3, 50, 89]), np.array([], np.int64)]], [16])


def test_eviction_of_a_very_long_cache(T):
    """Ids and byte offsets far out: 17 million tokens, rows beyond 4 GiB."""
    ctx, budget = 17_000_000, 1000
    s = make(T, 1, 1, 1, 64, ctx, bs=2048)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.rand((1, 1, ctx), generator=g, device="cuda")
    far = torch.randperm(ctx, generator=g, device="cuda")[:budget - 20].sort().values
    w[0, 0, far] += 2 + torch.rand(budget - 20, generator=g, device="cuda")
    rows = torch.randint(0, 256, (1, 1, ctx, 256), generator=g, device="cuda", dtype=torch.uint8)  # 4.4 GB
    keep, new = torch.zeros((1, 1, budget), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    T.tls_evict_select(s, budget, 4, 16, w, i32([ctx]), keep, new)
    torch.cuda.synchronize()
    got = keep[0, 0].long()
    must = torch.cat((torch.arange(4, device="cuda"), far, torch.arange(ctx - 16, ctx, device="cuda"))).unique()
    assert new.item() == budget and (got[1:] > got[:-1]).all() and torch.isin(must, got).all()
    want, ww, tail = rows[0, 0, got].clone(), w[0, 0, got].clone(), rows[0, 0, -5000:].clone()
    T.tls_evict_compact(s, budget, keep, i32([ctx]), [rows], w)
    torch.cuda.synchronize()
    assert torch.equal(rows[0, 0, :budget], want) and torch.equal(rows[0, 0, -5000:], tail)
    assert torch.equal(w[0, 0, :budget], ww) and not w[0, 0, budget:].any()


# --------------------------------------------------------------------------------------- used together
def test_decode_loop_over_a_4bit_cache_with_eviction(T):
    """A prompt into the 4-bit cache, decode steps that append a token, select, attend and add up weights, and an
    eviction whenever the cache is full, followed by a rebuilt summary.  Every step's attention and weights are
    held to the 64-bit forms on the values that the mirror on the host says are stored."""
    rng = np.random.default_rng(42)
    B, H, G, d, ctx, bs, r, kb, kt = 2, 2, 4, 64, 160, 16, 16, 6, 48
    budget, sink, recent = 96, 2, 24
    s = T.make_shape(batch=B, n_q_heads=H * G, n_kv_heads=H, d_qk=d, d_v=d, block_size=bs, n_label=r, k_b=kb, k_t=kt,
                     max_ctx=ctx, kv_dtype=T.TLS_BF16)
    nb = ctx // bs
    dev = dict(device="cuda")
    cache = torch.zeros((B, H, ctx, 9 * d // 8), dtype=torch.uint8, **dev)
    meta, slab = torch.zeros((B, H, nb, 2, d), dtype=BF16, **dev), torch.zeros((B, H, ctx, r), dtype=BF16, **dev)
    label = i32(sorted(rng.permutation(d)[:r].tolist()))
    w = torch.zeros((B, H, ctx), **dev)
    ws = torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, **dev)
    bidx, tidx = torch.zeros((B, H, kb), dtype=torch.int32, **dev), torch.zeros((B, H, kt), dtype=torch.int32, **dev)
    out, lse = torch.zeros((B, H * G, d), **dev), torch.zeros((B, H * G), **dev)
    keep, tmp = torch.zeros((B, H, budget), dtype=torch.int32, **dev), torch.zeros((B,), dtype=torch.int32, **dev)
    rows = lambda n: torch.from_numpy(rng.standard_normal((B, H, n, d)).astype(np.float32)).to(BF16)
    mirror = np.zeros((B, H, ctx, 9 * d // 8), np.uint8)
    mirror_w = np.zeros((B, H, ctx))
    lens = [140, 97]
    prompt = rows(140), rows(140)
    old, new = i32([0, 0]), i32(lens)
    T.tls_kv4_append(s, prompt[0].cuda(), prompt[1].cuda(), old, new, 140, cache, label, meta, slab)
    rec = R.records(f64(prompt[0]), f64(prompt[1]))
    for b in range(B):
        mirror[b, :, :lens[b]] = rec[b, :, :lens[b]]
    evictions = 0
    for step in range(70):
        if max(lens) == ctx:  # full: evict, move, rebuild the summary from the stored keys
            T.tls_evict_select(s, budget, sink, recent, w, new, keep, tmp)
            T.tls_evict_compact(s, budget, keep, new, [cache, slab], w)
            acc = w.cpu().numpy()
            for b in range(B):
                for h in range(H):
                    k = R.keep(got_w[b, h], lens[b], budget, sink, recent)
                    np.testing.assert_array_equal(keep[b, h, :len(k)].cpu().numpy(), k)
                    mirror[b, h, :len(k)] = mirror[b, h, k]
                    mirror_w[b, h, :len(k)] = mirror_w[b, h, k]
                    mirror_w[b, h, len(k):] = 0
                    np.testing.assert_array_equal(acc[b, h, :len(k)], got_w[b, h, k])
                    assert (acc[b, h, len(k):] == 0).all()
                lens[b] = min(lens[b], budget)
            new = tmp.clone()
            K = torch.zeros((B, H, ctx, d), dtype=BF16, **dev)
            T.tls_kv4_read(s, cache, torch.zeros_like(new), new, ctx, K)
            T.tls_build_block_meta(s, K, new, label, meta, None)
            evictions += 1
        old, new = new, new + 1
        k1, v1 = rows(1), rows(1)
        T.tls_kv4_append(s, k1.cuda(), v1.cuda(), old, new, 1, cache, label, meta, slab)
        rec = R.records(f64(k1), f64(v1))
        for b in range(B):
            mirror[b, :, lens[b]] = rec[b, :, 0]
            lens[b] += 1
        q = torch.from_numpy(rng.standard_normal((B, H * G, d)).astype(np.float32)).to(BF16)
        qd = q.cuda()
        T.tls_select_step(s, qd, meta, slab, label, new, bidx, tidx)
        T.tls_kv4_attn_decode(s, qd, cache, out, lse, token_idx=tidx, ws=ws)
        T.tls_kv4_accum_weights(s, qd, cache, lse, w, token_idx=tidx)
        torch.cuda.synchronize()
        assert T.tls_device_error(clear=True) == 0
        tk, got_w = tidx.cpu().numpy(), w.cpu().numpy()
        for b in range(B):
            for h in range(H):
                t = tk[b, h][tk[b, h] >= 0]
                assert len(t) == min(kt, lens[b]) and (np.diff(t) > 0).all() and t.max() < lens[b]
                K, V = R.split(mirror[b, h], d)
                hs = slice(h * G, (h + 1) * G)
                wo, wl, tol, ltol = R.attention(f64(q[b, hs]), K, V, t, 1 / np.sqrt(d))
                assert (np.abs(f64(out[b, hs]) - wo) <= tol).all() and (np.abs(f64(lse[b, hs]) - wl) <= ltol).all()
                add, wtol = R.weights(f64(q[b, hs]), K, f64(lse[b, hs]), t, 1 / np.sqrt(d), ctx)
                prev = mirror_w[b, h].copy()
                mirror_w[b, h] = got_w[b, h]
                assert (np.abs(got_w[b, h] - (prev + add)) <= wtol + R.U32 * (prev + add)).all()
    assert evictions >= 1 and (mirror[:, :, :min(lens)] == cache.cpu().numpy()[:, :, :min(lens)]).mean() > 0.999


def test_captured_upkeep_replays(T):
    """Append, attention, weights, selection and compaction captured in one graph and replayed on new inputs give the
    bits of the eager calls."""
    rng = np.random.default_rng(5)
    B, H, G, d, ctx, budget = 2, 2, 4, 64, 1200, 700
    s = make(T, B, H, G, d, ctx)
    start = torch.from_numpy(R.records(rng.standard_normal((B, H, ctx, d)), rng.standard_normal((B, H, ctx, d)))).cuda()
    w_start = torch.rand((B, H, ctx), device="cuda")
    K, V, q = (torch.zeros(sh, dtype=BF16, device="cuda") for sh in ((B, H, 1, d), (B, H, 1, d), (B, H * G, d)))
    old, new = i32([1100, 900]), i32([1101, 901])
    ws = torch.empty(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda")
    cache, w = start.clone(), w_start.clone()
    out, lse = torch.zeros((B, H * G, d), device="cuda"), torch.zeros((B, H * G), device="cuda")
    keep, lens = torch.zeros((B, H, budget), dtype=torch.int32, device="cuda"), i32([0, 0])
    back = torch.zeros((B, H, ctx, d), dtype=BF16, device="cuda")

    def step():
        T.tls_kv4_append(s, K, V, old, new, 1, cache)
        T.tls_kv4_attn_decode(s, q, cache, out, lse, seq_lens=new, ws=ws)
        T.tls_kv4_accum_weights(s, q, cache, lse, w, seq_lens=new)
        T.tls_evict_select(s, budget, 4, 32, w, new, keep, lens)
        T.tls_evict_compact(s, budget, keep, new, [cache], w)
        T.tls_kv4_read(s, cache, i0, lens, ctx, back)

    i0 = i32([0, 0])

    def fresh(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for x in (K, V, q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        cache.copy_(start)
        w.copy_(w_start)
        for x in (out, lse, keep, lens, back):
            x.zero_()

    def outputs():
        torch.cuda.synchronize()
        return [x.clone() for x in (cache, w, out, lse, keep, lens, back)]

    want = []
    for seed in (1, 2):
        fresh(seed)
        step()
        want.append(outputs())
    graph = torch.cuda.CUDAGraph()
    fresh(3)
    with torch.cuda.graph(graph):
        step()
    for seed, ref in ((2, want[1]), (1, want[0]), (2, want[1])):
        fresh(seed)
        graph.replay()
        for a, b in zip(outputs(), ref):
            assert torch.equal(a, b)
    assert T.tls_device_error(clear=True) == 0


def test_compact_weights_alone(T):
    s = make(T, 1, 2, 1, 64, 50)
    w0 = torch.rand((1, 2, 50), device="cuda") + 1
    w = w0.clone()
    keep = i32([[[1, 4, 30, -1], [0, 1, 2, 44]]])
    T.tls_evict_compact(s, 4, keep, i32([45]), [], w)
    want = w0.clone()
    want[:, :, :45] = 0
    want[0, 0, :3], want[0, 1, :4] = w0[0, 0, [1, 4, 30]], w0[0, 1, [0, 1, 2, 44]]
    assert torch.equal(w, want)


def late_gaps(rng, B, H, lens, budget):
    """Kept ids that are the identity for a while, then ever sparser: rows move by little, then by much."""
    keeps = []
    for n in lens:
        per_head = []
        for _ in range(H):
            k = min(n, budget)
            head = k // 2 if n > budget else k
            rest = np.sort(rng.permutation(np.arange(head, n))[:k - head])
            per_head.append(np.concatenate([np.arange(head), rest]))
        keeps.append(per_head)
    return keeps


@pytest.mark.parametrize("offset,rows,ctx,budget", [(0, [256, 256], 3000, 1500), (1, [256], 1100, 500), (2, [256, 32], 1100, 500),
                                                    (0, [144], 3000, 2900)])
def test_compact_many_groups_over_several_chunks(T, offset, rows, ctx, budget):
    """64 groups and more: each slice is moved by one large CTA, chunk after chunk, a chunk's stores directly before
    the next one's loads (256 rows a chunk with 16-byte accesses, 16 with single bytes)."""
    rng = np.random.default_rng(offset + len(rows))
    B, H = (8, 8) if len(rows) > 1 else (16, 8)
    lens = [ctx, ctx - 1, ctx // 2, budget, budget + 1, 1, 0, ctx] * (B // 8)
    for keeps in (late_gaps(rng, B, H, lens, budget), random_keeps(rng, B, H, lens, budget)):
        run_compact(T, B, H, ctx, lens, budget, keeps, rows, offset=offset)


def test_stored_values_and_summary_over_evictions(T):
    """Prompt, eviction, rebuilt summary, appended tokens, again and again: every live row holds exactly the values of
    its token (only the sign of a zero may differ), the rebuilt summary is the max / min of the stored keys, and
    appended rows enter it as given."""
    rng = np.random.default_rng(11)
    B, H, d, ctx, bs, budget = 2, 3, 128, 260, 32, 130
    s = make(T, B, H, 1, d, ctx, bs=bs)
    nb = -(-ctx // bs)
    dev = dict(device="cuda")
    cache = torch.zeros((B, H, ctx, 9 * d // 8), dtype=torch.uint8, **dev)
    meta, label = torch.zeros((B, H, nb, 2, d), dtype=BF16, **dev), i32(list(range(16)))
    w = torch.zeros((B, H, ctx), **dev)
    keep, tmp = torch.zeros((B, H, budget), dtype=torch.int32, **dev), torch.zeros((B,), dtype=torch.int32, **dev)
    lens = [0, 0]
    K_at, V_at = np.zeros((B, H, ctx, d)), np.zeros((B, H, ctx, d))  # the values stored at each row
    K_sum = np.zeros((B, H, ctx, d))  # the keys that the summary knows: as given, or as stored since the last rebuild

    def check():
        torch.cuda.synchronize()
        got = cache.cpu().numpy()
        m = f64(meta)
        for b in range(B):
            n = lens[b]
            gk, gv = R.split(got[b, :, :n], d)
            np.testing.assert_array_equal(gk, K_at[b, :, :n])
            np.testing.assert_array_equal(gv, V_at[b, :, :n])
            for blk in range(-(-n // bs)):
                part = K_sum[b, :, blk * bs:min(n, (blk + 1) * bs)]
                np.testing.assert_array_equal(m[b, :, blk, 0], part.max(1))
                np.testing.assert_array_equal(m[b, :, blk, 1], part.min(1))

    def append(counts):
        n = max(counts)
        rows = [torch.from_numpy(rng.standard_normal((B, H, n, d)).astype(np.float32)).to(BF16) for _ in range(2)]
        old, new = i32(lens), i32([a + c for a, c in zip(lens, counts)])
        T.tls_kv4_append(s, rows[0].cuda(), rows[1].cuda(), old, new, n, cache, label, meta, None)
        K, V = (R.value(*R.quantise(f64(x))) for x in rows)
        for b in range(B):
            K_at[b, :, lens[b]:lens[b] + counts[b]], V_at[b, :, lens[b]:lens[b] + counts[b]] = K[b, :, :counts[b]], V[b, :, :counts[b]]
            K_sum[b, :, lens[b]:lens[b] + counts[b]] = f64(rows[0])[b, :, :counts[b]]
            lens[b] += counts[b]

    append([250, 131])
    check()
    for turn in range(3):
        w.copy_(torch.from_numpy(heavy(rng, (B, H, ctx))))
        T.tls_evict_select(s, budget, 4, 20, w, i32(lens), keep, tmp)
        T.tls_evict_compact(s, budget, keep, i32(lens), [cache], w)
        ids = keep.cpu().numpy()
        for b in range(B):
            for h in range(H):
                k = ids[b, h][ids[b, h] >= 0]
                assert len(k) == min(lens[b], budget)
                K_at[b, h, :len(k)], V_at[b, h, :len(k)] = K_at[b, h, k], V_at[b, h, k]
            lens[b] = min(lens[b], budget)
        K = torch.zeros((B, H, ctx, d), dtype=BF16, **dev)
        T.tls_kv4_read(s, cache, torch.zeros_like(tmp), tmp, ctx, K)
        T.tls_build_block_meta(s, K, tmp, label, meta, None)
        K_sum[:] = K_at
        check()
        append([1, 1])
        check()
        append([100 - turn, 37])
        check()
    assert T.tls_device_error(clear=True) == 0
