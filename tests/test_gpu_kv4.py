"""The 4-bit KV cache on the GPU: rows in and out (bit-exact against the 64-bit quantiser, the summary and slab
against a full build) and the attention over it, in every form the header names, against the 64-bit attention
over the stored values (bounds: tests/_kv4.py)."""
import numpy as np
import pytest
import torch

from tests import _kv4 as R
from two_level_sparse_quest_b200 import workloads as W

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


def shape(T, B, H, G, d, ctx, bs=32, kt=64, out=0, r=16):
    return T.make_shape(batch=B, n_q_heads=H * G, n_kv_heads=H, d_qk=d, d_v=d, block_size=bs, n_label=r,
                        k_b=1, k_t=kt, max_ctx=ctx, kv_dtype=T.TLS_BF16, out_dtype=out)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16_rows(rng, shape, scale=1.0, outliers=True):
    x = rng.standard_normal(shape).astype(np.float32) * scale
    if outliers:
        x[..., 3::shape[-1] // 8] *= 5
    return torch.from_numpy(x).to(BF16)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


# ------------------------------------------------------------------------------------------- rows in, out
STORE = {
    # name: (B, H, d, ctx, bs, old, new, row_stride)
    "prompt_d128": (2, 2, 128, 300, 32, [0, 0], [300, 171], 300),
    "prompt_d64_odd": (3, 1, 64, 77, 16, [0, 0, 0], [77, 1, 0], 77),
    "one_token_mid_block": (3, 2, 128, 100, 32, [40, 63, 64], [41, 64, 65], 1),
    "one_token_from_empty": (1, 1, 64, 9, 4, [0], [1], 1),
    "ragged_over_blocks": (2, 3, 128, 333, 7, [5, 100], [300, 133], 295),
    "block_of_one": (1, 2, 64, 150, 1, [10], [150], 140),
    "one_block_of_all": (1, 1, 128, 700, 1024, [3], [700], 700),
    "wider_rows_than_needed": (2, 1, 128, 64, 32, [0, 60], [5, 64], 50),
}


@pytest.mark.parametrize("name", sorted(STORE))
def test_append_and_read(T, name):
    B, H, d, ctx, bs, old, new, stride = STORE[name]
    rng = np.random.default_rng(11)
    s = shape(T, B, H, 4, d, ctx, bs)
    Kall, Vall = bf16_rows(rng, (B, H, ctx, d)), bf16_rows(rng, (B, H, ctx, d), 0.02, False)
    rows = [torch.full((B, H, stride, d), 7.0, dtype=BF16) for _ in range(2)]
    for b in range(B):
        for dst, src in zip(rows, (Kall, Vall)):
            dst[b, :, :new[b] - old[b]] = src[b, :, old[b]:new[b]]
    assert T.tls_kv4_cache_bytes(s) == B * H * ctx * 9 * d // 8
    cache = torch.full((B, H, ctx, 9 * d // 8), 0xA5, dtype=torch.uint8, device="cuda")
    label = i32(sorted(rng.permutation(d)[:16].tolist()))
    nb = -(-ctx // bs)

    def built(lens):
        meta = torch.zeros((B, H, nb, 2, d), dtype=BF16, device="cuda")
        slab = torch.zeros((B, H, ctx, 16), dtype=BF16, device="cuda")
        T.tls_build_block_meta(s, Kall.cuda(), i32(lens), label, meta, slab)
        return meta, slab

    meta, slab = built(old)
    T.tls_kv4_append(s, rows[0].cuda(), rows[1].cuda(), i32(old), i32(new), stride, cache, label, meta, slab)
    want_meta, want_slab = built(new)
    outs = [torch.full((B, H, stride, d), 9.0, dtype=BF16, device="cuda") for _ in range(2)]
    T.tls_kv4_read(s, cache, i32(old), i32(new), stride, *outs)
    only_v = torch.full((B, H, stride, d), 9.0, dtype=BF16, device="cuda")
    T.tls_kv4_read(s, cache, i32(old), i32(new), stride, None, only_v)
    torch.cuda.synchronize()
    assert T.tls_device_error(clear=True) == 0
    assert torch.equal(meta.view(torch.int16), want_meta.view(torch.int16))
    assert torch.equal(slab.view(torch.int16), want_slab.view(torch.int16))
    assert torch.equal(only_v, outs[1])
    got = cache.cpu().numpy()
    want = R.records(f64(Kall), f64(Vall))
    h, c = d // 2, d // 16
    for b in range(B):
        live = slice(old[b], new[b])
        np.testing.assert_array_equal(got[b, :, live, h:h + 2 * c], want[b, :, live, h:h + 2 * c])  # scales
        for x, y, o in zip(R.split(got[b, :, live], d), R.split(want[b, :, live], d), outs):
            np.testing.assert_array_equal(x, y)
            np.testing.assert_array_equal(f64(o[b, :, :new[b] - old[b]]), y)  # exact in bf16
            assert (o[b, :, new[b] - old[b]:] == 9).all()
        assert (got[b, :, :old[b]] == 0xA5).all() and (got[b, :, new[b]:] == 0xA5).all()


def test_append_special_values(T):
    """Ties, zeros, the smallest and largest groups, clamping, infinities and NaN (whole groups read as NaN)."""
    d, n = 128, 16
    x = np.zeros((n, d), np.float32)
    x[0, :16] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, 0]
    x[0, 16:32] = x[0, :16] * 1.125          # ties of a scale that is no power of two
    x[0, 32:48] = x[0, :16] * 1.75 * 2.0 ** -9
    x[1, :16] = 1e-7                          # scale 0
    x[1, 16:32] = np.linspace(-2.0 ** -17 * 7, 2.0 ** -17 * 7, 16)  # the smallest scales
    x[1, 32:48] = np.linspace(-2e-4, 2e-4, 16)
    x[2, :16] = np.linspace(-61440, 61440, 16)
    x[2, 16:32] = np.linspace(-3e38, 3e38, 16)  # clamped
    x[3, 5], x[3, 20], x[3, 40] = np.inf, -np.inf, np.nan
    x[3, 6], x[3, 21], x[3, 100] = 1, 2, 3
    x[4, :] = -0.0
    x[5:] = np.random.default_rng(3).standard_normal((n - 5, d)) * np.exp2(np.arange(n - 5) * 3 - 18)[:, None]
    K = torch.from_numpy(x).to(BF16)[None, None]
    s = shape(T, 1, 1, 1, d, n)
    cache = torch.zeros((1, 1, n, 144), dtype=torch.uint8, device="cuda")
    T.tls_kv4_append(s, K.cuda(), K.flip(2).contiguous().cuda(), i32([0]), i32([n]), n, cache)
    out = [torch.zeros((1, 1, n, d), dtype=BF16, device="cuda") for _ in range(2)]
    T.tls_kv4_read(s, cache, i32([0]), i32([n]), n, *out)
    code, b = R.quantise(f64(K))
    want = R.value(code, b)
    np.testing.assert_array_equal(f64(out[0]), want)
    np.testing.assert_array_equal(f64(out[1]), want[:, :, ::-1])
    assert np.isnan(want[0, 0, 3, :48]).all() and want[0, 0, 3, 100] == 3 and np.abs(want[0, 0, 2]).max() == 61440


def test_append_refuses_bad_ranges_on_the_device(T):
    s = shape(T, 4, 1, 1, 64, 32)
    cache = torch.full((4, 1, 32, 72), 1, dtype=torch.uint8, device="cuda")
    rows = torch.ones((4, 1, 8, 64), dtype=BF16, device="cuda")
    out = torch.zeros_like(rows)
    bad = (i32([5, -1, 0, 30]), i32([4, 3, 9, 33]))  # new < old, old < 0, longer than row_stride, beyond max_ctx
    T.tls_device_error(clear=True)
    T.tls_kv4_append(s, rows, rows, *bad, 8, cache)
    torch.cuda.synchronize()
    assert T.tls_device_error(clear=True) == 4 and (cache == 1).all()
    T.tls_kv4_read(s, cache, *bad, 8, out)
    torch.cuda.synchronize()
    assert T.tls_device_error(clear=True) == 4 and (out == 0).all()


# --------------------------------------------------------------------------------------------- attention
def check_attention(T, B, H, G, d, ctx, tokens, mode, out_dtype=0, bs=32, seed=5, qscale=1.0, slots=None, softmax_scale=None):
    """tokens: [B][H] lists (with -1 and ids beyond the context among them), or per-sequence lengths (mode dense)."""
    rng = np.random.default_rng(seed)
    kt = 1 if mode == "dense" else len(tokens[0][0])
    s = shape(T, B, H, G, d, ctx, bs, kt, out_dtype)
    if softmax_scale:
        s.softmax_scale = softmax_scale
    q = bf16_rows(rng, (B, H * G, d), qscale, False)
    rec = R.records(f64(bf16_rows(rng, (B, H, ctx, d))), f64(bf16_rows(rng, (B, H, ctx, d), 1.0, False)))
    out = torch.full((B, H * G, d), 7.0, dtype=BF16 if out_dtype else torch.float32, device="cuda")
    lse = torch.full((B, H * G), 7.0, device="cuda")
    ws = torch.full((T.tls_kv4_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    kw = {}
    cache = rec
    if mode == "dense":
        kw["seq_lens"] = i32(tokens)
        tokens = [[list(range(n))] * H for n in tokens]
    else:
        kw["token_idx"] = i32(tokens)
    resident = None
    if mode == "paged":
        nb = -(-ctx // bs)
        n_slots = slots or nb
        table = np.full((B, H, nb), -1, np.int32)
        cache = rng.integers(0, 256, (B, H, n_slots, bs, rec.shape[-1]), dtype=np.uint8)
        for b in range(B):
            for h in range(H):
                for i, blk in enumerate(rng.permutation(nb)[:n_slots]):
                    slot = (i * 7 + 3) % n_slots if n_slots % 7 else i
                    table[b, h, blk] = slot
                    part = rec[b, h, blk * bs:(blk + 1) * bs]
                    cache[b, h, slot, :len(part)] = part
        resident = table
        if nb > 2:
            table[:, :, 0] = n_slots  # out of range: treated as not resident
        kw["slot_of_block"], kw["n_slots"] = torch.from_numpy(table).cuda(), n_slots
    T.tls_kv4_attn_decode(s, q.cuda(), torch.from_numpy(np.ascontiguousarray(cache)).cuda(), out, lse, ws=ws, **kw)
    torch.cuda.synchronize()
    assert T.tls_device_error(clear=True) == 0
    o, ls = f64(out), f64(lse)
    tau = softmax_scale or 1 / np.sqrt(d)
    for b in range(B):
        for h in range(H):
            K, V = R.split(rec[b, h], d)
            t = [x for x in tokens[b][h] if 0 <= x < ctx]
            if resident is not None:
                t = [x for x in t if 0 <= resident[b, h, x // bs] < kw["n_slots"]]
            hs = slice(h * G, (h + 1) * G)
            wo, wl, tol, ltol = R.attention(f64(q[b, hs]), K, V, t, tau)
            if out_dtype:  # half a step of fp16 on every weight, half a step of bf16 on the result
                p = np.exp(f64(q[b, hs]) @ K[t].T * tau - wl[:, None]) if len(t) else np.zeros((G, 0))
                tol = tol + 2.0 ** -11 * (p @ np.abs(V[t]))
                tol = tol + 2.0 ** -8 * (np.abs(wo) + tol)
            over = float((np.abs(o[b, hs] - wo) / tol).max())
            assert over <= 1, (b, h, over)
            fin = np.isfinite(wl)
            assert (np.isneginf(ls[b, hs]) == ~fin).all()
            assert (np.abs(ls[b, hs][fin] - wl[fin]) <= ltol[fin]).all()


def lists(rng, B, H, ctx, kt, pad=0, sort=True):
    t = np.full((B, H, kt), -1, np.int64)
    for b in range(B):
        for h in range(H):
            n = min(kt - pad, ctx)
            x = rng.permutation(ctx)[:n]
            t[b, h, :n] = np.sort(x) if sort else x
    return t.tolist()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 32, 64])
def test_attention_heads(T, d, G):
    rng = np.random.default_rng(G)
    check_attention(T, 2, 2 if G < 16 else 1, G, d, 500, lists(rng, 2, 2 if G < 16 else 1, 500, 131, pad=3), "list")


@pytest.mark.parametrize("kt", [1, 2, 15, 16, 17, 31, 32, 33, 64, 255, 256, 257, 511, 1000])
def test_attention_list_lengths(T, kt):
    rng = np.random.default_rng(kt)
    check_attention(T, 1, 2, 4, 128, 1024, lists(rng, 1, 2, 1024, kt, sort=kt % 2 == 0), "list", out_dtype=kt % 2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[0, 1, 31], [32, 33, 255], [256, 257, 999], [0, 0, 0]])
def test_attention_dense_lengths(T, d, lens):
    check_attention(T, 3, 1, 4, d, 999, lens, "dense", out_dtype=1)  # odd capacity: records at 8-byte offsets (d 64)


@pytest.mark.parametrize("d,bs,slots", [(128, 32, None), (64, 16, 9), (128, 7, 30), (64, 1, None)])
def test_attention_paged(T, d, bs, slots):
    rng = np.random.default_rng(bs)
    check_attention(T, 2, 2, 4, d, 301, lists(rng, 2, 2, 301, 200), "paged", bs=bs, slots=slots)


def test_attention_masked_ids(T):
    """-1 anywhere in the list, ids beyond the context, repeated ids, and a list with nothing valid."""
    bad = [-1, 5, -7, 99, 5, 100, 2 ** 31 - 1, 0] + [-1] * 40 + [98, -1, 7]
    none = [-1] * len(bad)
    check_attention(T, 1, 3, 8, 128, 100, [[bad, none, [100] * len(bad)]], "list")


def test_attention_few_groups_split_over_clusters(T):
    """One group over a long cache: several clusters, joined by the second launch; also where parts are empty."""
    check_attention(T, 1, 1, 4, 64, 30011, [30011], "dense")
    check_attention(T, 2, 1, 16, 128, 12000, [12000, 40], "dense", out_dtype=1)
    rng = np.random.default_rng(2)
    check_attention(T, 1, 1, 2, 128, 9000, lists(rng, 1, 1, 9000, 8193, pad=5000), "list")


@pytest.mark.parametrize("qscale", [1e-30, 1e-3, 30.0, 1e30])
def test_attention_query_range(T, qscale):
    """Queries far outside fp16, and a softmax that one token wins."""
    rng = np.random.default_rng(7)
    check_attention(T, 1, 2, 4, 128, 400, lists(rng, 1, 2, 400, 300), "list", qscale=qscale,
                    softmax_scale=min(1 / np.sqrt(128), 20 / qscale) if qscale > 1 else None)


def test_attention_small_weights_add_up(T):
    """One token ahead of 20000 others by 18 (natural log): their weights of 2^-26 still count together."""
    d, n = 128, 20001
    K, V = np.zeros((n, d)), np.zeros((n, d))
    K[:, 0], V[:, 0] = 6.0, 1.0
    K[77, 0], V[77, 0] = -6.0, -1.0
    rec = R.records(K, V)[None, None]
    q = torch.zeros((1, 1, d), dtype=BF16)
    q[0, 0, 0] = -1.5
    s = shape(T, 1, 1, 1, d, n)
    s.softmax_scale = 1.0
    out = torch.zeros((1, 1, d), device="cuda")
    T.tls_kv4_attn_decode(s, q.cuda(), torch.from_numpy(rec).cuda(), out, seq_lens=i32([n]),
                          ws=torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda"))
    wo, _, tol, _ = R.attention(f64(q[0]), *R.split(rec[0, 0], d), range(n), 1.0)  # the stored values
    assert abs(out[0, 0, 0].item() - wo[0, 0]) <= tol[0, 0]
    alone, _, _, _ = R.attention(f64(q[0]), *R.split(rec[0, 0], d), [77], 1.0)
    assert abs(wo[0, 0] - alone[0, 0]) > 5 * 2.0 ** -39 * n  # the small weights are far above what is dropped


def test_attention_nan_stays_where_it_is(T):
    """A NaN record that no list names changes nothing; one that is named makes its group NaN, as does a NaN query."""
    rng = np.random.default_rng(9)
    d, ctx, H, G = 128, 200, 3, 4
    K, V = rng.standard_normal((1, H, ctx, d)), rng.standard_normal((1, H, ctx, d))
    rec = R.records(K, V)
    s = shape(T, 1, H, G, d, ctx, kt=40)
    tok = np.sort(rng.permutation(ctx - 1)[:40])[None, None].repeat(H, 1)
    q = bf16_rows(rng, (1, H * G, d), 1.0, False)
    ws = torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda")

    def run(rec, q=q):
        out, lse = torch.zeros((1, H * G, d), device="cuda"), torch.zeros((1, H * G), device="cuda")
        T.tls_kv4_attn_decode(s, q.cuda(), torch.from_numpy(rec).cuda(), out, lse, token_idx=i32(tok.tolist()), ws=ws)
        return out.cpu(), lse.cpu()

    out, lse = run(rec)
    hidden = rec.copy()
    unused = np.setdiff1d(np.arange(ctx), tok[0, 0])
    hidden[:, :, unused] = 0xFF
    out2, lse2 = run(hidden)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    seen = rec.copy()
    seen[0, 1, tok[0, 1, 33], d // 2] = 0xFF  # a K scale of group 1
    out3, lse3 = run(seen)
    assert out3[0, G:2 * G].isnan().all() and lse3[0, G:2 * G].isnan().all()
    assert torch.equal(out3[0, :G], out[0, :G]) and torch.equal(out3[0, 2 * G:], out[0, 2 * G:])
    seen = rec.copy()
    seen[0, 2, tok[0, 2, 0], d // 2 + d // 16] = 0xFF  # a V scale of group 2: its 16 channels
    out4, lse4 = run(seen)
    assert out4[0, 2 * G:, :16].isnan().all() and torch.equal(out4[0, 2 * G:, 16:], out[0, 2 * G:, 16:])
    assert torch.equal(lse4, lse)
    qn = q.clone()
    qn[0, 2, 5] = float("nan")
    out5, lse5 = run(rec, qn)
    assert out5[0, 2].isnan().all() and lse5[0, 2].isnan() and torch.equal(out5[0, 3:], out[0, 3:])
    qn[0, 2, 5] = float("inf")  # scores of +-inf: NaN, as inf - inf
    out6, _ = run(rec, qn)
    assert out6[0, 2].isnan().all() and torch.equal(out6[0, 3:], out[0, 3:]) and torch.equal(out6[0, :2], out[0, :2])


def test_attention_on_a_stream_and_in_a_graph(T):
    """Another stream; a captured call replayed on new inputs; two graphs that share a workspace, one after the
    other; the same bits each time."""
    rng = np.random.default_rng(1)
    d, ctx, B, H, G = 64, 12000, 1, 1, 4  # few groups: the call that uses its workspace
    s = shape(T, B, H, G, d, ctx)
    rec = torch.from_numpy(R.records(rng.standard_normal((B, H, ctx, d)), rng.standard_normal((B, H, ctx, d)))).cuda()
    q = [bf16_rows(rng, (B, H * G, d), 1.0, False).cuda() for _ in range(2)]
    lens = i32([ctx])
    ws = torch.empty(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda")
    want = []
    for x in q:
        o = torch.zeros((B, H * G, d), device="cuda")
        T.tls_kv4_attn_decode(s, x, rec, o, seq_lens=lens, ws=ws)
        want.append(o)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = torch.zeros_like(want[0])
    side.wait_stream(torch.cuda.current_stream())
    T.tls_kv4_attn_decode(s, q[0], rec, o, seq_lens=lens, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0])
    buf, outs, graphs = q[0].clone(), [], []
    for _ in range(2):
        g, o = torch.cuda.CUDAGraph(), torch.zeros_like(want[0])
        with torch.cuda.graph(g):
            T.tls_kv4_attn_decode(s, buf, rec, o, seq_lens=lens, ws=ws)
        graphs.append(g)
        outs.append(o)
    for i in (1, 0):
        buf.copy_(q[i])
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[i]) and torch.equal(outs[1], want[i])


@pytest.mark.parametrize("kscale,vscale", [(2e-4, 1e-4), (1.0, 1e-4), (3e-5, 20000.0), (100.0, 1.0)])
def test_attention_of_small_and_large_rows(T, kscale, vscale):
    """Scales down to the smallest (values that are subnormal in fp16) and up to the clamp."""
    rng = np.random.default_rng(13)
    d, ctx, H, G = 128, 300, 2, 4
    rec = R.records(rng.standard_normal((1, H, ctx, d)) * kscale, rng.standard_normal((1, H, ctx, d)) * vscale)
    s = shape(T, 1, H, G, d, ctx)
    s.softmax_scale = 0.3 / kscale
    q = bf16_rows(rng, (1, H * G, d), 0.2, False)
    out, lse = torch.zeros((1, H * G, d), device="cuda"), torch.zeros((1, H * G), device="cuda")
    T.tls_kv4_attn_decode(s, q.cuda(), torch.from_numpy(rec).cuda(), out, lse, seq_lens=i32([ctx]),
                          ws=torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda"))
    for h in range(H):
        hs = slice(h * G, (h + 1) * G)
        wo, wl, tol, ltol = R.attention(f64(q[0, hs]), *R.split(rec[0, h], d), range(ctx), float(s.softmax_scale))
        assert (np.abs(f64(out[0, hs]) - wo) <= tol).all() and (np.abs(f64(lse[0, hs]) - wl) <= ltol).all()


def test_rows_beyond_4_gib(T):
    """Records whose byte offsets pass 32 bits: stored, read back, attended and weighed."""
    d, ctx = 128, 31_000_000
    s = shape(T, 1, 1, 4, d, ctx, bs=2048, kt=40)
    cache = torch.zeros((1, 1, ctx, 144), dtype=torch.uint8, device="cuda")  # 4.5 GB
    rng = np.random.default_rng(21)
    n, first = 50, ctx - 50
    K, V = bf16_rows(rng, (1, 1, n, d)), bf16_rows(rng, (1, 1, n, d), 1.0, False)
    T.tls_kv4_append(s, K.cuda(), V.cuda(), i32([first]), i32([ctx]), n, cache)
    out = torch.zeros((1, 1, n, d), dtype=BF16, device="cuda")
    T.tls_kv4_read(s, cache, i32([first]), i32([ctx]), n, out)
    code, b = R.quantise(f64(K))
    np.testing.assert_array_equal(f64(out), R.value(code, b))
    assert (cache[0, 0, :first].view(-1, 144)[-1000:] == 0).all() and (cache[0, 0, 0] == 0).all()
    rec = R.records(f64(K), f64(V))[0, 0]
    tok = np.sort(rng.permutation(n)[:40])
    q = bf16_rows(rng, (1, 4, d), 1.0, False)
    o, lse = torch.zeros((1, 4, d), device="cuda"), torch.zeros((1, 4), device="cuda")
    T.tls_kv4_attn_decode(s, q.cuda(), cache, o, lse, token_idx=i32([[(tok + first).tolist()]]),
                          ws=torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda"))
    Kv, Vv = R.split(rec, d)
    wo, wl, tol, _ = R.attention(f64(q[0]), Kv, Vv, tok, 1 / np.sqrt(d))
    assert (np.abs(f64(o[0]) - wo) <= tol).all()
    w = torch.zeros((1, 1, ctx), device="cuda")
    T.tls_kv4_accum_weights(s, q.cuda(), cache, lse, w, token_idx=i32([[(tok + first).tolist()]]))
    add, wtol = R.weights(f64(q[0]), Kv, f64(lse[0]), tok, 1 / np.sqrt(d), n)
    assert (np.abs(f64(w[0, 0, first:]) - add) <= wtol + 4 * R.U32 * add).all() and (w[0, 0, :first] == 0).all()


@pytest.mark.parametrize("d,bs", [(128, 32), (128, 7), (64, 16)])
def test_prefetched_blocks_are_attended(T, d, bs):
    """A stream of selections over 4-bit blocks in pinned host memory: each step copies the blocks that entered,
    and the attention over the slot cache gives the bits of the attention over the whole cache."""
    rng = np.random.default_rng(bs)
    B, H, G, ctx, kb = 2, 2, 4, 40 * bs - 3, 6
    nb, kt, rb = -(-ctx // bs), 3 * bs, 9 * d // 8
    n_slots = 2 * kb
    s = T.make_shape(batch=B, n_q_heads=H * G, n_kv_heads=H, d_qk=d, d_v=d, block_size=bs, n_label=16, k_b=kb, k_t=kt,
                     max_ctx=ctx, kv_dtype=T.TLS_BF16)
    rec = R.records(rng.standard_normal((B, H, ctx, d)), rng.standard_normal((B, H, ctx, d)))
    host = torch.zeros((B, H, nb * bs, rb), dtype=torch.uint8).pin_memory()
    host[:, :, :ctx] = torch.from_numpy(rec)
    whole = torch.from_numpy(rec).cuda()
    dev = dict(dtype=torch.int32, device="cuda")
    cache = torch.full((B, H, n_slots, bs, rb), 0xFF, dtype=torch.uint8, device="cuda")
    sob, bos = torch.empty((B, H, nb), **dev), torch.empty((B, H, n_slots), **dev)
    n_new, jobs = torch.empty((B, H), **dev), torch.empty((B, H, kb, 2), **dev)
    ws = torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda")
    T.tls_offload_reset(s, n_slots, sob, bos)
    prev, held, resident = None, [[set() for _ in range(H)] for _ in range(B)], [[set() for _ in range(H)] for _ in range(B)]
    for step in range(6):
        sel = [[rng.permutation(sorted(held[b][h]))[:3].astype(int).tolist() for h in range(H)] for b in range(B)]
        for b in range(B):
            for h in range(H):
                rest = [x for x in rng.permutation(nb).tolist() if x not in sel[b][h]]
                sel[b][h] = sorted(sel[b][h] + rest[:kb - len(sel[b][h])])
        nxt = i32(sel)
        T.tls_kv4_prefetch_diff(s, n_slots, host, cache, sob, bos, prev, nxt, n_new, jobs)
        tok = np.full((B, H, kt), -1)
        for b in range(B):
            for h in range(H):
                cand = np.concatenate([np.arange(x * bs, min((x + 1) * bs, ctx)) for x in sel[b][h]])
                pick = np.sort(rng.permutation(cand)[:kt])
                tok[b, h, :len(pick)] = pick
        q = bf16_rows(rng, (B, H * G, d), 1.0, False).cuda()
        outs = [torch.zeros((B, H * G, d), device="cuda") for _ in range(2)]
        T.tls_kv4_attn_decode(s, q, cache, outs[0], token_idx=i32(tok.tolist()), slot_of_block=sob, n_slots=n_slots, ws=ws)
        T.tls_kv4_attn_decode(s, q, whole, outs[1], token_idx=i32(tok.tolist()), ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and outs[0].isfinite().all()
        for b in range(B):
            for h in range(H):
                # a block stays resident while the previous or the next selection holds it
                assert n_new[b, h].item() == len(set(sel[b][h]) - resident[b][h])
                resident[b][h] = held[b][h] | set(sel[b][h])
                held[b][h] = set(sel[b][h])
        prev = nxt
    assert T.tls_device_error(clear=True) == 0


def test_attention_many_groups_and_clamped_lengths(T):
    rng = np.random.default_rng(17)
    check_attention(T, 70, 3, 2, 64, 60, lists(rng, 70, 3, 60, 35, pad=1), "list", out_dtype=1)
    check_attention(T, 2, 1, 32, 128, 9001, [9001, 4500], "dense", out_dtype=1)  # two units a group, cut into parts
    # lengths outside [0, max_ctx] are clamped: compared with the clamped ones
    d, ctx = 128, 333
    s = shape(T, 3, 1, 4, d, ctx)
    rec = torch.from_numpy(R.records(rng.standard_normal((3, 1, ctx, d)), rng.standard_normal((3, 1, ctx, d)))).cuda()
    q = bf16_rows(rng, (3, 4, d), 1.0, False).cuda()
    ws = torch.zeros(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda")
    got = []
    for lens in ([-3, 2 ** 31 - 1, 5], [0, ctx, 5]):
        out, lse = torch.full((3, 4, d), 7.0, device="cuda"), torch.full((3, 4), 7.0, device="cuda")
        T.tls_kv4_attn_decode(s, q, rec, out, lse, seq_lens=i32(lens), ws=ws)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not got[0][0][0].any() and (got[0][1][0] == -float("inf")).all()


def test_summary_of_special_values(T):
    """Signed zeros, infinities, NaN and a column that holds nothing else: the summary's bits are a full build's,
    whether the rows come at once or one by one."""
    d, n, bs = 64, 24, 8
    x = np.random.default_rng(2).standard_normal((n, d)).astype(np.float32)
    x[:, 0], x[::2, 1], x[1::2, 1] = np.nan, 0.0, -0.0
    x[:, 2], x[5, 3], x[6, 3], x[7, 4] = -0.0, np.inf, -np.inf, np.nan
    K = torch.from_numpy(x).to(BF16)[None, None].cuda()
    s = shape(T, 1, 1, 2, d, n, bs)
    label = i32(list(range(16)))
    want = [torch.zeros((1, 1, n // bs, 2, d), dtype=BF16, device="cuda"), torch.zeros((1, 1, n, 16), dtype=BF16, device="cuda")]
    T.tls_build_block_meta(s, K, i32([n]), label, *want)
    for step in (n, 5, 1):
        got = [torch.zeros_like(w) for w in want]
        cache = torch.zeros((1, 1, n, 72), dtype=torch.uint8, device="cuda")
        for t in range(0, n, step):
            e = min(n, t + step)
            rows = K[:, :, t:e].contiguous()
            T.tls_kv4_append(s, rows, rows, i32([t]), i32([e]), e - t, cache, label, *got)
        for g, w in zip(got, want):
            assert torch.equal(g.view(torch.int16), w.view(torch.int16)), step


@pytest.mark.parametrize("d,G,out", [(64, 1, 0), (64, 1, 1), (64, 2, 0), (128, 1, 1)])
def test_attention_few_outputs_shared_by_a_cluster(T, d, G, out):
    """One or two heads over a list that takes a cluster of eight: a CTA's share of the joined outputs is less than a
    warp, so some lanes only of one warp write between the cluster's barriers."""
    rng = np.random.default_rng(d + G)
    check_attention(T, 1, 2, G, d, 2500, lists(rng, 1, 2, 2500, 2300, pad=100), "list", out_dtype=out)
    check_attention(T, 1, 1, G, d, 2500, [2500], "dense", out_dtype=out)


def both_outputs(T, B, H, G, d, ctx, kw, kt=64, bs=32, cache=None, seed=0):
    """The same call with an fp32 and with a bf16 output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((B, H * G, d), generator=g, device="cuda").to(BF16)
    res = []
    for out in (0, 1):
        s = shape(T, B, H, G, d, ctx, bs=bs, kt=kt, out=out)
        o = torch.zeros((B, H * G, d), dtype=BF16 if out else torch.float32, device="cuda")
        lse = torch.zeros((B, H * G), device="cuda")
        ws = torch.empty(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda")
        T.tls_kv4_attn_decode(s, q, cache, o, lse, ws=ws, **kw)
        res.append((o, lse))
    return res


@pytest.mark.parametrize("d,G", [(64, 1), (64, 16), (128, 4), (128, 8), (128, 16), (128, 64)])
@pytest.mark.parametrize("mode", ["list", "paged", "dense"])
def test_attention_output_type_rounds_the_result_only(T, mode, d, G):
    """A bf16 output is the fp32 output rounded once: the softmax weights carry the same bits for both."""
    rng = np.random.default_rng(G)
    B, H, ctx, bs, kt = 2, 2, 3000, 16, 1500
    rec = torch.from_numpy(R.records(rng.standard_normal((B, H, ctx, d)), rng.standard_normal((B, H, ctx, d)))).cuda()
    kw = dict(seq_lens=i32([ctx, 777]))
    if mode != "dense":
        kw = dict(token_idx=i32(lists(rng, B, H, ctx, kt, pad=3)))
    if mode == "paged":
        nb = -(-ctx // bs)
        rec = torch.cat((rec, rec[:, :, :nb * bs - ctx]), 2).contiguous()
        kw.update(slot_of_block=torch.arange(nb, dtype=torch.int32, device="cuda").expand(B, H, nb).contiguous(), n_slots=nb)
    (o32, l32), (o16, l16) = both_outputs(T, B, H, G, d, ctx, kw, kt=kt, bs=bs, cache=rec)
    assert torch.equal(l32, l16) and o32.isfinite().all() and o32.any()
    assert torch.equal(o32.to(BF16), o16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 8, 16, 32, 64])
def test_attention_heads_over_long_lists_and_slots(T, d, G):
    """Lists of a few thousand tokens (clusters or parts), bf16 output, over the cache and over a slot cache of which
    some blocks are missing."""
    rng = np.random.default_rng(d + G)
    ctx, kt = 4100, 3001
    H = 2 if G < 16 else 1
    check_attention(T, 1, H, G, d, ctx, lists(rng, 1, H, ctx, kt, pad=7), "list", out_dtype=1)
    check_attention(T, 1, H, G, d, ctx, lists(rng, 1, H, ctx, kt, pad=7), "paged", bs=16, slots=200, out_dtype=G > 4)
    check_attention(T, 2, H, G, d, 400, lists(rng, 2, H, 400, 131), "paged", bs=32, out_dtype=G <= 4)


@pytest.mark.parametrize("d,G,out", [(64, 64, 0), (128, 32, 0), (128, 64, 1), (64, 32, 1), (128, 16, 0)])
def test_attention_many_heads_over_a_long_cache(T, d, G, out):
    """Every token of 20001, in several units of 16 heads and many parts; a short sequence beside it."""
    check_attention(T, 2, 1, G, d, 20001, [20001, 33], "dense", out_dtype=out)


def test_attention_calls_at_once(T):
    """Calls on several streams at the same time, each with its own workspace and output, give the bits of calls one
    after another."""
    rng = np.random.default_rng(3)
    B, H, G, d, ctx = 1, 2, 4, 128, 20000
    rec = torch.from_numpy(R.records(rng.standard_normal((B, H, ctx, d)), rng.standard_normal((B, H, ctx, d)))).cuda()
    s = shape(T, B, H, G, d, ctx, kt=2000)
    tok, lens = i32(lists(rng, B, H, ctx, 2000)), i32([ctx])
    n = 4
    q = [bf16_rows(rng, (B, H * G, d), 1.0, False).cuda() for _ in range(n)]
    ws = [torch.empty(T.tls_kv4_workspace_size(s), dtype=torch.uint8, device="cuda") for _ in range(n)]

    def run(i, out, w, stream=None):
        kw = dict(token_idx=tok) if i % 2 else dict(seq_lens=lens)
        T.tls_kv4_attn_decode(s, q[i], rec, out, ws=ws[i], stream=stream, **kw)
        T.tls_kv4_accum_weights(s, q[i], rec, torch.zeros((B, H * G), device="cuda"), w, stream=stream, **kw)

    outs = [[torch.zeros((B, H * G, d), device="cuda") for _ in range(n)] for _ in range(2)]
    sums = [[torch.zeros((B, H, ctx), device="cuda") for _ in range(n)] for _ in range(2)]
    for i in range(n):
        run(i, outs[0][i], sums[0][i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(n)]
    for i in range(n):
        with torch.cuda.stream(streams[i]):
            run(i, outs[1][i], sums[1][i])
    torch.cuda.synchronize()
    for i in range(n):
        assert torch.equal(outs[0][i], outs[1][i]) and torch.equal(sums[0][i], sums[1][i])
