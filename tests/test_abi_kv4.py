"""Host-side checks of the 4-bit cache and the eviction entry points (no GPU: every refusal comes before a launch),
and the 64-bit test forms themselves against hand-worked values."""
import ctypes

import numpy as np
import pytest

from tests import _kv4 as R


@pytest.fixture(scope="module")
def T():
    from two_level_sparse_quest_b200 import build

    build.build()
    from two_level_sparse_quest_b200 import tls

    return tls


def good(T, **kw):
    base = dict(batch=2, n_q_heads=32, n_kv_heads=8, d_qk=128, d_v=128, block_size=32, n_label=16, k_b=64, k_t=512,
                max_ctx=4096, kv_dtype=T.TLS_BF16)
    base.update(kw)
    return T.make_shape(**base)


def latent(T, **kw):
    return good(T, v_is_k_prefix=True, n_q_heads=64, n_kv_heads=1, d_qk=576, d_v=512, **kw)


def by(s):
    return ctypes.byref(s)


def append(T, s, K=256, V=256, old=256, new=256, stride=4, label=256, cache=256, meta=256, slab=256):
    return T._lib.tls_kv4_append(by(s), K, V, old, new, stride, label, cache, meta, slab, None)


def read(T, s, cache=256, old=256, new=256, stride=4, K=256, V=256):
    return T._lib.tls_kv4_read(by(s), cache, old, new, stride, K, V, None)


def attn(T, s, q=256, cache=256, tok=256, lens=256, slots=None, n_slots=0, out=256, lse=256, ws=256, n=1 << 40):
    return T._lib.tls_kv4_attn_decode(by(s), q, cache, tok, lens, slots, n_slots, out, lse, ws, n, None)


def test_kv4_shapes(T):
    s = good(T)
    assert T.tls_kv4_cache_bytes(s) == 2 * 8 * 4096 * 144
    assert T.tls_kv4_cache_bytes(good(T, d_qk=64, d_v=64)) == 2 * 8 * 4096 * 72
    assert T.tls_kv4_workspace_size(s) % 256 == 0 and T.tls_kv4_workspace_size(s) >= 256
    assert T.tls_kv4_cache_bytes(good(T, batch=0)) == 0
    for bad, word in ((good(T, kv_dtype=T.TLS_F32), "bf16"), (latent(T), "GQA")):
        for call in (append, read, attn):
            assert call(T, bad) == T.TLS_ERR_UNSUPPORTED and word in T.tls_last_error()
        st = T._lib.tls_kv4_accum_weights(by(bad), 256, 256, 256, None, 256, 256, None)
        assert st == T.TLS_ERR_UNSUPPORTED
        with pytest.raises(T.TlsError):
            T.tls_kv4_cache_bytes(bad)
        with pytest.raises(T.TlsError):
            T.tls_kv4_workspace_size(bad)
    assert attn(T, good(T, n_q_heads=24)) == T.TLS_ERR_UNSUPPORTED  # 3 heads per group


def test_kv4_rows_refusals(T):
    s = good(T)
    for kw, word in ((dict(K=None), "K is NULL"), (dict(V=None), "V is NULL"), (dict(K=264), "aligned"),
                     (dict(cache=None), "cache is NULL"), (dict(cache=260), "aligned"), (dict(old=None), "old_lens"),
                     (dict(new=257), "new_lens"), (dict(stride=-1), "row_stride"), (dict(stride=4097), "row_stride"),
                     (dict(label=None), "label_idx"), (dict(meta=264), "meta"), (dict(slab=264), "slab")):
        assert append(T, s, **kw) == T.TLS_ERR_INVALID_ARG and word in T.tls_last_error(), kw
    q8 = good(T, slab_bits=8)
    assert append(T, q8) == T.TLS_ERR_UNSUPPORTED and "int8" in T.tls_last_error()
    for kw, word in ((dict(K=None, V=None), "both NULL"), (dict(K=264), "K_out"), (dict(V=264), "V_out"),
                     (dict(stride=5000), "row_stride"), (dict(cache=None), "cache is NULL")):
        assert read(T, s, **kw) == T.TLS_ERR_INVALID_ARG and word in T.tls_last_error(), kw
    # nothing to do: no pointer is looked at
    assert append(T, s, stride=0, K=None, V=None, cache=None) == T.TLS_OK
    assert read(T, good(T, batch=0), cache=None, K=None, V=None) == T.TLS_OK


def test_kv4_attention_refusals(T):
    s = good(T)
    need = T.tls_kv4_workspace_size(s)
    for kw, word in ((dict(q=None), "q is NULL"), (dict(cache=8), "aligned"), (dict(tok=None, lens=None), "seq_lens"),
                     (dict(tok=258), "token_idx"), (dict(out=None), "out is NULL"), (dict(out=264), "out"),
                     (dict(lse=258), "lse_out"), (dict(slots=256, n_slots=0), "n_slots"), (dict(slots=258, n_slots=4), "slot_of_block")):
        assert attn(T, s, **kw) == T.TLS_ERR_INVALID_ARG and word in T.tls_last_error(), kw
    assert attn(T, s, tok=None, slots=256, n_slots=4) == T.TLS_ERR_UNSUPPORTED and "token_idx" in T.tls_last_error()
    assert attn(T, s, slots=256, n_slots=2 ** 27) == T.TLS_ERR_UNSUPPORTED and "int32" in T.tls_last_error()
    for kw in (dict(ws=None), dict(n=need - 1), dict(ws=0x1010)):
        assert attn(T, s, **kw) == T.TLS_ERR_WORKSPACE and str(need) in T.tls_last_error()
    assert attn(T, good(T, batch=0), q=None, cache=None, out=None, ws=None) == T.TLS_OK


def test_kv4_prefetch_refusals(T):
    call = lambda s, n=384, host=256, cache=256, prev=None, nxt=256: T._lib.tls_kv4_prefetch_diff(
        by(s), n, host, cache, 256, 256, prev, nxt, 256, 256, None)
    s = good(T)
    for kw, word in ((dict(n=0), "n_slots"), (dict(n=5000), "n_slots"), (dict(host=None), "host_kv"),
                     (dict(cache=264), "cache"), (dict(prev=258), "prev_block_idx"), (dict(nxt=None), "next_block_idx")):
        assert call(s, **kw) == T.TLS_ERR_INVALID_ARG and word in T.tls_last_error(), kw
    assert call(good(T, kv_dtype=T.TLS_F32)) == T.TLS_ERR_UNSUPPORTED
    assert call(good(T, d_qk=64, d_v=64, block_size=7)) == T.TLS_ERR_UNSUPPORTED and "even" in T.tls_last_error()
    assert call(good(T, batch=0), host=None, cache=None, nxt=None) == T.TLS_OK


def test_lists_beyond_int_are_refused(T):
    s = good(T, k_t=2 ** 30 + 1)
    assert attn(T, s) == T.TLS_ERR_UNSUPPORTED and "k_t" in T.tls_last_error()
    assert T._lib.tls_accum_weights(by(s), 256, 256, 256, None, 256, 256, None) == T.TLS_ERR_UNSUPPORTED


def test_accum_weights_refusals(T):
    call = lambda s, q=256, K=256, tok=256, lens=256, lse=256, w=256: T._lib.tls_accum_weights(by(s), q, K, tok, lens, lse, w, None)
    s = good(T)
    for kw, word in ((dict(q=None), "q is NULL"), (dict(K=264), "keys"), (dict(tok=None, lens=None), "seq_lens"),
                     (dict(lse=None), "lse is NULL"), (dict(w=None), "weights is NULL"), (dict(w=258), "weights")):
        assert call(s, **kw) == T.TLS_ERR_INVALID_ARG and word in T.tls_last_error(), kw
    assert call(good(T, d_qk=96, d_v=96)) == T.TLS_ERR_UNSUPPORTED
    assert call(good(T, batch=0), None, None, None, None, None, None) == T.TLS_OK


def test_evict_refusals(T):
    s = good(T)
    sel = lambda s=s, budget=100, sink=4, recent=8, w=256, lens=256, keep=256, new=512: T._lib.tls_evict_select(
        by(s), budget, sink, recent, w, lens, keep, new, None)
    for kw, word in ((dict(budget=0), "budget"), (dict(budget=4097), "budget"), (dict(sink=-1), "n_sink"),
                     (dict(recent=-1), "n_recent"), (dict(sink=50, recent=51), "fit the budget"),
                     (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), "fit the budget"), (dict(w=None), "weights is NULL"),
                     (dict(lens=None), "seq_lens is NULL"), (dict(keep=None), "keep_idx_out is NULL"),
                     (dict(new=None), "new_lens_out is NULL"), (dict(new=256), "overlaps"), (dict(new=260), "overlaps")):
        assert sel(**kw) == T.TLS_ERR_INVALID_ARG and word in T.tls_last_error(), kw
    assert sel(good(T, batch=0), w=None, lens=None, keep=None, new=None) == T.TLS_OK

    def comp(ptrs=(1 << 30,), sizes=(256,), s=s, budget=100, keep=256, lens=256, w=None, n=None):
        n = len(ptrs) if n is None else n
        m = max(1, len(ptrs))
        return T._lib.tls_evict_compact(by(s), budget, keep, lens, n, (ctypes.c_void_p * m)(*ptrs),
                                        (ctypes.c_int32 * m)(*sizes), w, None)

    for kw, word in ((dict(budget=0), "budget"), (dict(n=9), "n_rows"), (dict(n=-1), "n_rows"),
                     (dict(ptrs=(None,)), "rows[0] is NULL"), (dict(sizes=(0,)), "row_bytes[0]"),
                     (dict(sizes=(65537,)), "row_bytes[0]"), (dict(keep=None), "keep_idx is NULL"),
                     (dict(lens=None), "seq_lens is NULL"), (dict(w=258), "weights"),
                     (dict(ptrs=(1 << 30, (1 << 30) + 2 * 8 * 4096 * 16 - 1), sizes=(16, 16)), "overlap"),
                     (dict(w=(1 << 30) + 4), "overlap")):
        assert comp(**kw) == T.TLS_ERR_INVALID_ARG and word in T.tls_last_error(), kw
    st = T._lib.tls_evict_compact(by(s), 100, 256, 256, 1, None, None, None, None)
    assert st == T.TLS_ERR_INVALID_ARG and "rows" in T.tls_last_error()
    assert comp(ptrs=(), sizes=(), keep=None, lens=None) == T.TLS_OK  # nothing to move
    assert comp(s=good(T, batch=0), keep=None, lens=None) == T.TLS_OK


def test_binding_refuses_host_tensors_and_wrong_row_shapes(T):
    import torch

    s = good(T)
    cpu = torch.zeros(16, dtype=torch.int32)
    for f in (lambda: T.tls_kv4_append(s, cpu, 256, 256, 256, 1, 256), lambda: T.tls_kv4_read(s, 256, 256, 256, 1, cpu),
              lambda: T.tls_kv4_attn_decode(s, 256, cpu, 256, seq_lens=256, ws=(256, 1 << 30)),
              lambda: T.tls_accum_weights(s, 256, 256, cpu, 256, seq_lens=256),
              lambda: T.tls_kv4_accum_weights(s, 256, 256, 256, cpu, seq_lens=256),
              lambda: T.tls_evict_select(s, 10, 1, 1, 256, 256, cpu, 512)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    with pytest.raises(ValueError, match="max_ctx"):
        T.tls_evict_compact(s, 10, 256, 256, [torch.zeros((2, 8, 4095, 4))])


def test_quantiser_of_the_tests_by_hand():
    x = np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, 0.0])
    code, b = R.quantise(x)
    assert b.tolist() == [15 << 3]  # scale 1
    assert R.value(code, b).tolist() == [6, 4, 4, 2, 2, 1, 1, 0, -4, -4, -2, -2, -1, -1, 0, 0]
    code, b = R.quantise(x * 2.0 ** -17)  # scale 2^-17, the smallest
    assert b.tolist() == [1] and (R.value(code, b) == R.value(*R.quantise(x)) * 2.0 ** -17).all()
    assert R.quantise(x * 2.0 ** -20)[1].tolist() == [0] and R.quantise(x * 1e9)[1].tolist() == [0xE2]
    assert len(R.SCALES) == 0xE3 and R.SCALES[-1] == 10240 and (np.diff(R.SCALES) > 0).all()
    half = (np.arange(0xE3, dtype=np.uint16) << 7).view(np.float16)
    assert (half.astype(np.float64) == R.SCALES).all()
    rng = np.random.default_rng(0)
    K, V = rng.standard_normal((5, 64)), rng.standard_normal((5, 64))
    rec = R.records(K, V)
    assert rec.shape == (5, 72)
    for got, want in zip(R.split(rec, 64), (K, V)):
        assert (got == R.value(*R.quantise(want))).all()
        step = np.repeat(np.abs(want).reshape(5, 4, 16).max(-1), 16, -1)
        assert (np.abs(got - want) <= step / 6 * 1.07).all()  # half the widest step (4 to 6), scale rounded by 1/16


def test_kept_ids_of_the_tests_by_hand():
    w = np.array([0.0, 3.0, 1.0, 1.0, 0.5, 9.0, np.nan, 0.0], np.float32)
    assert R.keep(w, 8, 4, 1, 1).tolist() == [0, 1, 5, 7]
    assert R.keep(w, 8, 5, 1, 1).tolist() == [0, 1, 2, 5, 7]  # 1.0 twice: the lower index
    assert R.keep(w, 8, 7, 0, 0).tolist() == [0, 1, 2, 3, 4, 5, 7]  # NaN goes first
    assert R.keep(w, 3, 4, 1, 1).tolist() == [0, 1, 2]


def test_an_empty_batch_moves_nothing(T):
    """batch 0: the arrays are empty, and an empty tensor's pointer is NULL."""
    import torch

    s = good(T, batch=0)
    st = T._lib.tls_evict_compact(by(s), 100, None, None, 2, (ctypes.c_void_p * 2)(None, None),
                                  (ctypes.c_int32 * 2)(256, 144), None, None)
    assert st == T.TLS_OK, T.tls_last_error()
    st = T._lib.tls_evict_compact(by(s), 100, None, None, 1, (ctypes.c_void_p * 1)(None), (ctypes.c_int32 * 1)(0), None, None)
    assert st == T.TLS_ERR_INVALID_ARG and "row_bytes[0]" in T.tls_last_error()
    assert torch.empty((0, 8, 4096, 144)).data_ptr() == 0
    T.tls_evict_compact(s, 100, None, None, [(0, 256)], None, stream=1)
