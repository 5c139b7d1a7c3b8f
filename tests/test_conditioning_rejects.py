"""The conditioning entry points reject bad arguments on the host, before anything is launched (CPU only)."""
import ctypes

import pytest
import torch

import sequence_parallelism_st_b200 as st

VP = ctypes.c_void_p
Q, K, QO, KO, TAB, POS, O, WS = (VP(x << 32) for x in range(1, 9))


def qk(q=Q, k=K, qo=QO, ko=KO, table=TAB, n_pos=8, pos=None, gamma=None, **kw):
    d = dict(size=ctypes.sizeof(st.st_qk_desc), n_tokens=8, h_q=4, h_k=2, D=72, dtype=st.ST_BF16, eps=1e-6)
    d.update(kw)
    return st._c["st_qk_norm_rope"](ctypes.byref(st.st_qk_desc(**d)), q, k, qo, ko, gamma, None, table, n_pos, pos, None)


def test_qk_norm_rope_rejects():
    assert st._c["st_qk_norm_rope"](None, Q, K, QO, KO, None, None, None, 0, None, None) == st.ST_ERR_NULL
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None)):
        assert qk(**kw) == st.ST_ERR_NULL, kw
    for kw in (dict(size=8), dict(n_tokens=0), dict(h_q=-1), dict(h_q=0, h_k=0), dict(D=0), dict(pos_period=-1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(pairing=2), dict(stride_q=280), dict(stride_k_out=136),
               dict(n_pos=0), dict(n_pos=7), dict(pos_period=8, n_pos=7),
               dict(n_tokens=1 << 30, pos_period=1, h_q=64, h_k=64)):
        assert qk(**kw) == st.ST_ERR_SHAPE, kw
    assert qk(dtype=5) == st.ST_ERR_DTYPE
    for D in (36, 20, 264):
        assert qk(D=D) == st.ST_ERR_UNSUPPORTED
    for kw in (dict(q=VP(Q.value + 8)), dict(ko=VP(KO.value + 2)), dict(stride_q=292), dict(table=VP(TAB.value + 8)),
               dict(pos=VP(POS.value + 2)), dict(gamma=VP(POS.value + 1))):
        assert qk(**kw) == st.ST_ERR_ALIGN, kw


def test_qk_norm_rope_overlaps():
    # rows of 8 tokens, Q 4 * 72 and K 2 * 72 channels
    row, e = 6 * 72, 2
    for kw in (dict(qo=VP(Q.value + 16)),                                  # shifted output
               dict(qo=Q, stride_q=4 * 72, stride_q_out=4 * 72 + 8),       # in place with another stride
               dict(qo=K), dict(ko=Q), dict(ko=QO),
               # K's columns begin inside Q's of the same rows
               dict(k=VP(Q.value + 16 * 9), qo=Q, stride_q=row, stride_q_out=row, stride_k=row)):
        assert qk(**kw) == st.ST_ERR_SHAPE, kw


def cross(fn="st_attn_cross", q=Q, k=K, v=K, o=O, ws=None, wsb=0, lse=None, desc={}, kv={}, own={}):
    d = dict(B=4, T=2, S=64, H=4, D=72, dtype=st.ST_BF16)
    d.update(desc)
    g = dict(size=ctypes.sizeof(st.st_kv_desc), n_sets=4, L=77, H_kv=2)
    dk, do = st.st_kv_desc(**{**g, **kv}), st.st_kv_desc(**{**g, **own})
    d = st.make_desc(**d)
    if fn == "st_attn_cross":
        return st._c[fn](ctypes.byref(d), ctypes.byref(dk), q, k, v, o, lse, ws, wsb, None)
    return st._c[fn](ctypes.byref(d), ctypes.byref(dk), ctypes.byref(do), q, k, v, k, v, o, lse, ws, wsb, None)


@pytest.mark.parametrize("fn", ["st_attn_cross", "st_attn_prefix"])
def test_attention_rejects(fn):
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(o=None)):
        assert cross(fn, **kw) == st.ST_ERR_NULL, kw
    for kw in (dict(kv=dict(size=4)), dict(kv=dict(n_sets=0)), dict(kv=dict(L=-1)), dict(kv=dict(H_kv=-1)),
               dict(kv=dict(stride_l=136)), dict(kv=dict(stride_l=-144)), dict(kv=dict(L=0, len=POS.value)),
               dict(kv=dict(offsets=POS.value, len=POS.value, n_rows=9)),
               dict(kv=dict(offsets=POS.value, mask=POS.value, n_rows=9)),
               dict(kv=dict(offsets=POS.value, n_rows=1 << 31)), dict(kv=dict(n_rows=5)),
               dict(desc=dict(kv_begin=0, kv_end=5)), dict(desc=dict(stride_s=280)), dict(desc=dict(B=0)),
               dict(desc=dict(S=1 << 30))):
        assert cross(fn, **kw) == st.ST_ERR_SHAPE, kw
    assert cross(fn, kv=dict(n_sets=3)) == st.ST_ERR_DIVISIBILITY
    assert cross(fn, kv=dict(H_kv=3), own=dict(H_kv=3)) == st.ST_ERR_DIVISIBILITY
    assert cross(fn, desc=dict(dtype=7)) == st.ST_ERR_DTYPE
    for kw in (dict(desc=dict(D=40)), dict(desc=dict(D=136, dtype=st.ST_F32)), dict(desc=dict(n_slices=2, slice=0)),
               dict(desc=dict(s_block=8, stride_sb=8 * 288 + 8, stride_t=1 << 20))):
        assert cross(fn, **kw) == st.ST_ERR_UNSUPPORTED, kw
    for kw in (dict(q=VP(Q.value + 8)), dict(o=VP(O.value + 8)), dict(k=VP(K.value + 2)), dict(v=VP(K.value + 2)),
               dict(desc=dict(stride_s=292)), dict(kv=dict(stride_l=148)), dict(kv=dict(stride_set=77 * 144 + 4)),
               dict(kv=dict(len=POS.value + 2)), dict(lse=VP(POS.value + 2)), dict(ws=VP(WS.value + 8), wsb=1 << 40)):
        assert cross(fn, **kw) == st.ST_ERR_ALIGN, kw


def ws_bytes(fn, desc, *kvs):
    d = dict(B=4, T=1, S=1, H=4, D=72, dtype=st.ST_BF16)
    d.update(desc)
    ks = [ctypes.byref(st.st_kv_desc(**{**dict(size=ctypes.sizeof(st.st_kv_desc), n_sets=4, L=77, H_kv=2), **k}))
          for k in kvs]
    return st._c[fn + "_workspace_bytes"](ctypes.byref(st.make_desc(**d)), *ks)


def test_workspace():
    """Few queries over many keys ask for a workspace; a short one is refused, none is accepted."""
    n = ws_bytes("st_attn_cross", {}, dict(L=20000))
    assert n > 0 and n % (4 * 4 * 73 * 4) == 0                       # whole parts of 16 rows of D values and an LSE
    assert ws_bytes("st_attn_cross", dict(S=20000), dict(L=20000)) == 0
    assert ws_bytes("st_attn_cross", {}, dict(L=64)) == 0
    assert ws_bytes("st_attn_cross", dict(D=40), dict(L=20000)) == 0
    assert cross(desc=dict(T=1, S=1), kv=dict(L=20000), ws=WS, wsb=n - 1) == st.ST_ERR_SHAPE
    # samples that share a prefix are packed; those that do not are not
    assert ws_bytes("st_attn_prefix", dict(B=64), dict(n_sets=1, L=300), dict(n_sets=64)) > 0
    assert ws_bytes("st_attn_prefix", dict(B=64, S=300), dict(n_sets=64, L=300), dict(n_sets=64)) == 0
    assert cross("st_attn_prefix", own=dict(H_kv=4)) == st.ST_ERR_SHAPE


def test_binding_checks():
    """The binding refuses what the library cannot see: dtypes, shapes, strides, devices."""
    q, k = torch.zeros(2, 1, 3, 4, 8), torch.zeros(2, 5, 2, 8)
    o = torch.zeros_like(q)
    def code(fn, *a, **kw):
        with pytest.raises(st.StattnError) as e:
            fn(*a, **kw)
        return e.value.code
    assert code(st.st_attn_cross, q, k, k, o) == st.ST_ERR_NULL                       # not on a GPU
    assert code(st.st_attn_cross, q, k, k.bfloat16(), o) == st.ST_ERR_DTYPE
    assert code(st.st_attn_cross, q, k, k[:, :4], o) == st.ST_ERR_SHAPE
    assert code(st.st_attn_cross, q, k[..., :4], k[..., :4], o) == st.ST_ERR_SHAPE
    assert code(st.st_attn_cross, q, k, k, o.bfloat16()) == st.ST_ERR_DTYPE
    assert code(st.st_attn_cross, q, k, k, torch.zeros(2, 1, 4, 3, 8).transpose(2, 3)) == st.ST_ERR_SHAPE
    assert code(st.st_attn_cross, q, k[:1].expand(2, 5, 2, 8), k[:1].expand(2, 5, 2, 8), o) == st.ST_ERR_SHAPE
    assert code(st.st_attn_cross, q, k, k, o, kv_len=torch.zeros(2)) == st.ST_ERR_DTYPE
    assert code(st.st_attn_cross, q, k, k, o, kv_len=torch.zeros(3, dtype=torch.int32)) == st.ST_ERR_SHAPE
    assert code(st.st_attn_cross, q, k, k, o, kv_mask=torch.zeros(2, 5)) == st.ST_ERR_DTYPE
    assert code(st.st_attn_cross, q, k, k, o, torch.zeros(5)) == st.ST_ERR_SHAPE
    x = torch.zeros(6, 2, 16)
    assert code(st.st_qk_norm_rope, x) == st.ST_ERR_NULL
    assert code(st.st_qk_norm_rope, None) == st.ST_ERR_NULL
    assert code(st.st_qk_norm_rope, x, x[:5]) == st.ST_ERR_SHAPE
    assert code(st.st_qk_norm_rope, x, x.bfloat16()) == st.ST_ERR_DTYPE
    assert code(st.st_qk_norm_rope, x.transpose(1, 2)) == st.ST_ERR_SHAPE
    assert code(st.st_qk_norm_rope, x[:1].expand(6, 2, 16)) == st.ST_ERR_SHAPE
    assert code(st.st_qk_norm_rope, x, q_gamma=torch.ones(15)) == st.ST_ERR_SHAPE
    assert code(st.st_qk_norm_rope, x, rope_table=torch.zeros(6, 16)) == st.ST_ERR_NULL
    assert code(st.st_qk_norm_rope, x, positions=torch.zeros(6, dtype=torch.int64)) == st.ST_ERR_DTYPE


def test_qk_norm_rope_rejects_rows_beyond_its_indices():
    assert qk(h_q=(1 << 30) // 72 + 1, k=None, ko=None, h_k=0, n_tokens=1) == st.ST_ERR_SHAPE
    assert qk(h_q=2 ** 31 - 1, h_k=2 ** 31 - 1, n_tokens=1, D=8) == st.ST_ERR_SHAPE


def test_single_queries_at_any_stride_are_rows():
    """Queries one per sample or frame are packed whatever lies between them: the workspace of the dense layout."""
    row = 4 * 72
    for fn, B, kv in (("st_attn_prefix", 64, [dict(n_sets=1, L=4096), dict(n_sets=64, L=60)]),
                      ("st_attn_cross", 64, [dict(n_sets=1, L=4096)])):
        for desc in (dict(), dict(T=1, stride_b=3 * row), dict(stride_b=5 * row, stride_t=8, stride_s=row)):
            assert ws_bytes(fn, dict(B=B, **desc), *kv) == ws_bytes(fn, dict(B=B), *kv) > 0, (fn, desc)
    kv = [dict(n_sets=2, L=4096), dict(n_sets=2, L=0)]
    dense = ws_bytes("st_attn_prefix", dict(B=2, T=30), *kv)
    assert ws_bytes("st_attn_prefix", dict(B=2, T=30, stride_t=3 * row), *kv) == dense > 0
    # overlapping rows are not taken for rows of a tile
    assert ws_bytes("st_attn_prefix", dict(B=64, stride_b=8), dict(n_sets=1, L=4096), dict(n_sets=64, L=60)) == 0


def test_binding_takes_packed_sets_of_no_rows():
    """Offsets over K of no rows describe sets without keys, with and without max_len (not a descriptor of L = 0)."""
    q, k = torch.zeros(2, 1, 3, 4, 8), torch.zeros(0, 2, 8)
    off = torch.zeros(3, dtype=torch.int32)
    for most in (None, 7):
        d = st._kv_desc("test", 8, q, k, k, None, off, None, most)
        assert d.L >= 1 and d.n_rows == 0 and d.n_sets == 2
        a = st.make_desc(2, 1, 3, 4, 8, st.ST_F32)
        assert st._c["st_attn_cross"](ctypes.byref(a), ctypes.byref(d), VP(Q.value + 2), None, None, O, None, None, 0,
                                      None) == st.ST_ERR_ALIGN       # (past the checks of the descriptor)


def test_workspace_bytes_of_tensors_off_the_gpu():
    q, k = torch.zeros(2, 1, 3, 4, 8), torch.zeros(2, 5, 2, 8)
    for call in (lambda: st.st_attn_cross_workspace_bytes(q, k), lambda: st.st_attn_prefix_workspace_bytes(q, k, k)):
        with pytest.raises(st.StattnError) as e:
            call()
        assert e.value.code == st.ST_ERR_NULL


@pytest.mark.parametrize("fn", ["st_attn_cross", "st_attn_prefix"])
def test_two_level_strides_are_taken_in_fp32(fn):
    """Token blocks and frame blocks of the sliced layouts: fp32 goes on to the next check, bf16 is refused."""
    row = 4 * 72
    for desc in (dict(s_block=8, stride_sb=8 * row + 8, stride_t=1 << 20),
                 dict(t_block=1, stride_tb=1 << 22, stride_b=1 << 16)):
        assert cross(fn, q=VP(Q.value + 2), desc=dict(desc, dtype=st.ST_F32)) == st.ST_ERR_ALIGN
        assert cross(fn, desc=desc) == st.ST_ERR_UNSUPPORTED
