"""Conditioning entry points where they can go wrong in ways that plain sizes and values do not show.

Tolerances and helpers are those of the parity tests of the same operators.
"""
import pytest
import torch

import sequence_parallelism_st_b200 as st
from test_gpu_conditioning import BF, F32, HEAD_DIMS, check_attn, rand, run_cross, run_prefix, sets_of

pytestmark = pytest.mark.gpu

# rows and row tiles of a work item, keys per step and steps whose K and V stay in shared memory
TILES = {32: (3, 96), 64: (3, 96), 72: (3, 80), 80: (3, 80), 96: (3, 64), 128: (2, 128)}


def first_blocks(cols, q_blocks, ctas):
    """(head, row block) of each block's first item where the items are cut evenly: heads and units outside,
    row blocks inside, as the launch does when there are more heads and units than blocks."""
    assert cols > ctas
    n = cols * q_blocks
    share = -(-n // ctas)
    assert share >= q_blocks                           # one band
    return [divmod(n * c // ctas, q_blocks) for c in range(ctas)]


@pytest.mark.parametrize("last", [100, 200])
@pytest.mark.parametrize("D", sorted(TILES))
def test_kept_keys_of_heads_that_share_them(D, last):
    """A block starts on the last rows of a head, where some of its row tiles have none, and goes on with a head
    of the same K and V, where they all have: every tile waits for the stages, which held NaN before."""
    nt, bn = TILES[D]
    last = min(last, (nt - 1) * 128)
    H, Hkv, ctas, full = 4, 1, 3, 2
    S, L = full * nt * 128 + last, 2 * bn - 7
    heads = first_blocks(H, full + 1, ctas)
    assert any(qb == full and h + 1 < H for h, qb in heads), heads
    assert -(-last // 128) < nt
    q, k, v = rand(200, 1, 1, S, H, D), rand(201, 1, L, Hkv, D), rand(202, 1, L, Hkv, D)
    poison = torch.full((148, L, 1, D), float("nan"), dtype=BF, device="cuda")
    qp = rand(203, 148, 1, nt * 128, 1, D)
    for _ in range(5):
        run_cross(qp, poison, poison)                  # every SM's stages hold NaN
        st.st_set_sm_budget(ctas)
        try:
            o, lse, _ = run_cross(q, k, v)
        finally:
            st.st_set_sm_budget(0)
        check_attn(q, [sets_of(k, v)], o, lse, what=f"D{D}")


NAN, INF = float("nan"), float("inf")


def nan_rows(o, lse, what):
    assert o.isnan().all() and lse.isnan().all(), what


def finite(o, lse, what):
    assert o.isfinite().all() and lse.isfinite().all(), what


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("L", [1, 4, 5, 300])
def test_values_that_are_not_finite_where_they_count(dtype, D, L):
    """NaN in a counted key, at every place of the 16 that are weighed together, early and late; NaN in one query;
    a score of +inf: the row's o and lse are NaN.  NaN and infinities of V reach their channel alone."""
    S, H = 5, 2
    q, k, v = rand(210, 1, 1, S, H, D, dtype=dtype), rand(211, 1, L, H, D, dtype=dtype), rand(212, 1, L, H, D, dtype=dtype)
    places = sorted({i for i in list(range(16)) + [L - 1 - i for i in range(16)] if 0 <= i < L})
    for i in places:
        kn = k.clone()
        kn[0, i, 0, D - 1] = NAN
        o, lse, _ = run_cross(q, kn, v)
        nan_rows(o[..., 0, :], lse[:, :, 0], f"K of key {i}")
        finite(o[..., 1, :], lse[:, :, 1], f"K of key {i}, the other head")
        vn = v.clone()
        vn[0, i, 0, 3], vn[0, i, 0, 5], vn[0, i, 1, 7] = NAN, INF, -INF
        o, lse, _ = run_cross(q, k, vn)
        assert lse.isfinite().all()
        assert o[..., 0, 3].isnan().all() and (o[..., 0, 5] == INF).all() and (o[..., 1, 7] == -INF).all()
        rest = o.clone()
        rest[..., 0, 3], rest[..., 0, 5], rest[..., 1, 7] = 0, 0, 0
        assert rest.isfinite().all(), f"V of key {i}"
        # a score beyond fp32: +inf
        big = torch.finfo(dtype).max / 4
        ko, qo = k.clone(), q.clone()
        ko[0, i, 1], qo[:, :, 2, 1] = big, 8.0
        qo[:, :, 3, 1] = -8.0                          # -inf for that key: a weight of 0, if another one counts
        o, lse, _ = run_cross(qo, ko, v)
        nan_rows(o[:, :, 2, 1], lse[:, :, 1, 2], f"+inf at key {i}")
        finite(o[:, :, :, 0], lse[:, :, 0], "the other head")
        if L > 1:
            finite(o[:, :, 3, 1], lse[:, :, 1, 3], f"-inf at key {i}")
        else:                                          # every score -inf: as a row without keys
            assert not o[:, :, 3, 1].any() and (lse[:, :, 1, 3] == -INF).all()
    for d in (0, D - 1):
        qn = q.clone()
        qn[0, 0, 2, 1, d] = NAN
        o, lse, _ = run_cross(qn, k, v)
        nan_rows(o[0, 0, 2, 1], lse[0, 0, 1, 2], "Q")
        o[0, 0, 2, 1], lse[0, 0, 1, 2] = 0, 0
        finite(o, lse, "the other rows")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [72, 128])
@pytest.mark.parametrize("S", [1, 40])
def test_values_that_are_not_finite_in_parts_and_prefixes(dtype, D, S):
    """The same where keys are split into parts, masked between, or attended behind a prefix (own keys in the
    combine kernel where samples are packed): one bad key that counts, in each part, makes the row NaN; one that
    does not leaves it finite."""
    B, H, Hkv, L = 2, 4, 2, 2000
    q, k, v = (rand(220 + i, *s, dtype=dtype) for i, s in enumerate([(B, 1, S, H, D), (B, L, Hkv, D), (B, L, Hkv, D)]))
    clean, clean_lse, ws = run_cross(q, k, v)
    assert ws > 0
    for i in (0, 5, 777, 1300, L - 1):
        kn = k.clone()
        kn[1, i, 1] = NAN
        o, lse, _ = run_cross(q, kn, v)
        nan_rows(o[1, :, :, 2:], lse[1, :, 2:], f"key {i}")
        assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :, :, :2], clean[1, :, :, :2])
        assert torch.equal(lse[0], clean_lse[0])
        keep = torch.ones(B, L, dtype=torch.bool)
        keep[1, i] = False
        o, lse, _ = run_cross(q, kn, v, kv_mask=keep.cuda())
        finite(o, lse, "masked")
    qn = q.clone()
    qn[0, 0, 0, 3, 1] = NAN
    o, lse, _ = run_cross(qn, k, v)
    nan_rows(o[0, 0, 0, 3], lse[0, 0, 3, 0], "Q")
    for B, sets, Lp, Lo in ((6, 2, 700, 9), (2, 2, 90, 150)):
        q = rand(223, B, 1, S, H, D, dtype=dtype)
        kp, vp = rand(224, sets, Lp, Hkv, D, dtype=dtype), rand(225, sets, Lp, Hkv, D, dtype=dtype)
        ko, vo = rand(226, B, Lo, Hkv, D, dtype=dtype), rand(227, B, Lo, Hkv, D, dtype=dtype)
        for ws in (True, False):
            for i in (0, 3, 4, Lo - 1):
                kn = ko.clone()
                kn[B - 1, i, 0, 1] = NAN
                o, lse, _ = run_prefix(q, kp, vp, kn, vo, ws=ws)
                nan_rows(o[B - 1, :, :, :2], lse[B - 1, :, :2], f"own key {i}")
                finite(o[:B - 1], lse[:B - 1], "the other samples")
                kn = kp.clone()
                kn[0, i % Lp, 1, 0] = NAN
                o, lse, _ = run_prefix(q, kn, vp, ko, vo, ws=ws)
                each = B // sets
                nan_rows(o[:each, :, :, 2:], lse[:each, :, 2:], f"prefix key {i}")
                finite(o[each:], lse[each:], "the other set")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 72), (2, 2, 128)])
def test_single_queries_at_a_stride(dtype, H, Hkv, D):
    """One query per sample, or per frame, out of rows that hold more: packed as dense ones are, with their bits,
    and what lies between the rows stays."""
    for B, T, sets, Lp, L in ((40, 1, 1, 900, 20), (6, 1, 2, 300, 300), (2, 25, 2, 700, 10), (1, 1, 1, 1500, 3)):
        q = rand(230, B, T, 1, H, D, dtype=dtype)
        wide = rand(231, B, T, 1, 3 * H, D, dtype=dtype)
        wide[..., :H, :] = q
        out, lse = torch.full_like(wide, 7.0), torch.empty(B, T, H, 1, device="cuda")
        kp, vp = rand(232, sets, Lp, Hkv, D, dtype=dtype), rand(233, sets, Lp, Hkv, D, dtype=dtype)
        k, v = rand(234, B, L, Hkv, D, dtype=dtype), rand(235, B, L, Hkv, D, dtype=dtype)
        for kw in (dict(), dict(kv_len=torch.arange(B, dtype=torch.int32).remainder(L + 1).cuda())):
            segs = [sets_of(kp, vp), sets_of(k, v, kw.get("kv_len"))]
            o, l, n = run_prefix(q, kp, vp, k, v, **kw)
            check_attn(q, segs, o, l, what="dense")
            assert st.st_attn_prefix_workspace_bytes(wide[..., :H, :], kp, k, **kw) == n
            for ws in (None, torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")):
                st.st_attn_prefix(wide[..., :H, :], kp, vp, k, v, out[..., :H, :], lse, workspace=ws, **kw)
                check_attn(q, segs, out[..., :H, :], lse, what="strided")
            assert torch.equal(out[..., :H, :], o) and torch.equal(lse, l)
        o, l, n = run_cross(q, kp, vp)
        assert st.st_attn_cross_workspace_bytes(wide[..., :H, :], kp) == n
        st.st_attn_cross(wide[..., :H, :], kp, vp, out[..., :H, :], lse, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert torch.equal(out[..., :H, :], o) and torch.equal(lse, l)
        assert (out[..., H:, :] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_len", [None, 5])
def test_packed_sets_of_no_rows(dtype, max_len):
    """Every prompt empty: K and V of no rows, with offsets: o = 0, lse = -inf, and nothing beside a prefix."""
    B, S, H, D = 3, 6, 2, 72
    q = rand(240, B, 1, S, H, D, dtype=dtype)
    e = torch.empty(0, H, D, dtype=dtype, device="cuda")
    off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    o, lse, _ = run_cross(q, e, e, kv_offsets=off, max_len=max_len)
    assert not o.any() and (lse == -INF).all()
    kp, vp = rand(241, 1, 70, H, D, dtype=dtype), rand(242, 1, 70, H, D, dtype=dtype)
    for ws in (True, False):
        o, lse, _ = run_prefix(q, kp, vp, e, e, ws=ws, kv_offsets=off, max_len=max_len)
        check_attn(q, [sets_of(kp, vp)], o, lse, what="no own keys")


@pytest.mark.parametrize("S,L,Lp", [(40, 33, 70), (2, 1500, 900), (130, 64, 1)])
@pytest.mark.parametrize("D", [72, 30])
def test_fp32_two_level_strides(S, L, Lp, D):
    """The sliced layout [token block, frame block, batch, frame, token, C] with gaps: Q and O found row by row, what
    lies between them left as it was."""
    B, T, H = 2, 4, 2
    nt, ns = 2, 2
    C, tf, ts = H * D, T // nt, S // ns
    big = rand(250, ns, nt, B, tf, ts + 3, C + 5, dtype=F32)
    dim = dict(zip(("ns", "nt", "b", "tf", "ts", "c"), big.stride()))
    desc = st.make_desc(B, T, S, H, D, st.ST_F32, stride_b=dim["b"], stride_t=dim["tf"], t_block=tf,
                        stride_tb=dim["nt"], stride_s=dim["ts"], s_block=ts, stride_sb=dim["ns"])

    def logical(x):
        return x[:, :, :, :, :ts, :C].permute(2, 1, 3, 0, 4, 5).reshape(B, T, S, H, D)
    k, v, kp, vp = (rand(251 + i, B if i < 2 else 1, n, H, D, dtype=F32) for i, n in enumerate((L, L, Lp, Lp)))
    q = logical(big)
    for fn, keys, segs in ((st.st_attn_cross, (k, v), [sets_of(k, v)]),
                           (st.st_attn_prefix, (kp, vp, k, v), [sets_of(kp, vp), sets_of(k, v)])):
        n = getattr(st, fn.__name__ + "_workspace_bytes")(big, *keys[::2], desc=desc)
        for ws in (None, torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")):
            out, lse = torch.full_like(big, 7.0), torch.full((B, T, H, S), NAN, device="cuda")
            fn(big, *keys, out, lse, workspace=ws, desc=desc)
            check_attn(q, segs, logical(out), lse, what=fn.__name__)
            assert (out[..., ts:, :] == 7.0).all() and (out[..., C:] == 7.0).all()


def time_of(f, n=3):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def budgeted(sms, f):
    st.st_set_sm_budget(sms)
    try:
        return f()
    finally:
        st.st_set_sm_budget(0)


@pytest.mark.parametrize("D", [40, 72, 128])
def test_fp32_within_the_budget(D):
    """The fp32 kernel on a few SMs: the bits of the whole GPU's run, and not on more SMs than it was given (one
    SM takes far longer than all)."""
    B, S, H, L = 3, 700, 4, 200
    q, k, v = rand(260, B, 1, S, H, D, dtype=F32), rand(261, B, L, H, D, dtype=F32), rand(262, B, L, H, D, dtype=F32)
    n = torch.tensor([L, 0, 77], dtype=torch.int32)
    o, lse, _ = run_cross(q, k, v, kv_len=n.cuda())
    check_attn(q, [sets_of(k, v, n)], o, lse, what="whole")
    for sms in (1, 5):
        o2, lse2, _ = budgeted(sms, lambda: run_cross(q, k, v, kv_len=n.cuda()))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    q, k, v = rand(263, 1, 1, 8192, 4, D, dtype=F32), rand(264, 1, L, 4, D, dtype=F32), rand(265, 1, L, 4, D, dtype=F32)
    out = torch.empty_like(q)
    def call():
        st.st_attn_cross(q, k, v, out)
    assert budgeted(1, lambda: time_of(call)) > 8 * time_of(call)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [72, 128])
@pytest.mark.parametrize("B,H,Hkv", [(40, 4, 2), (200, 8, 4)])
def test_combine_within_the_budget(dtype, D, B, H, Hkv):
    """Rows of split keys with own keys, joined by a few blocks (a warp and four warps a row): the same bits."""
    Lp, L = 900, 40
    n = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(270)).int()
    q = rand(271, B, 1, 1, H, D, dtype=dtype)
    kp, vp = rand(272, 1, Lp, Hkv, D, dtype=dtype), rand(273, 1, Lp, Hkv, D, dtype=dtype)
    k, v = rand(274, B, L, Hkv, D, dtype=dtype), rand(275, B, L, Hkv, D, dtype=dtype)
    o, lse, ws = run_prefix(q, kp, vp, k, v, kv_len=n.cuda())
    assert ws > 0
    check_attn(q, [sets_of(kp, vp), sets_of(k, v, n)], o, lse, what="whole")
    for sms in (1, 3):
        for _ in range(3):
            o2, lse2, _ = budgeted(sms, lambda: run_prefix(q, kp, vp, k, v, kv_len=n.cuda()))
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [72, 128])
@pytest.mark.parametrize("S", [100, 333])
@pytest.mark.parametrize("L", [2, 200])
def test_items_of_one_tile_with_kept_keys(D, S, L):
    """Row after row of queries with one set of keys and nothing to load but Q: at head dim 128 the loader runs up to
    four items ahead of a row tile, whose waits must all end (many short launches, items of one and two tiles)."""
    B, T, H, Hkv = 2, 3, 5, 1
    q = rand(280, B, T, S + 3, H, D)[:, :, :S]
    k, v = rand(281, B, L, Hkv, D), rand(282, B, L, Hkv, D)
    o, lse = torch.zeros(B, T, S + 3, H, D, dtype=BF, device="cuda")[:, :, :S], torch.empty(B, T, H, S, device="cuda")
    st.st_attn_cross(q, k, v, o, lse)
    assert st.st_check_device_status() == st.ST_OK
    check_attn(q, [sets_of(k, v)], o, lse, what="whole")
    for sms in (1, 3, 7, 11):
        o2, lse2 = torch.zeros(B, T, S + 3, H, D, dtype=BF, device="cuda")[:, :, :S], torch.empty_like(lse)
        for _ in range(100):
            budgeted(sms, lambda: st.st_attn_cross(q, k, v, o2, lse2))
        assert st.st_check_device_status() == st.ST_OK
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
