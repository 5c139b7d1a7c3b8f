"""Parity of the conditioning entry points against the fp64 oracle, element by element.

Tolerances, from the arithmetic (u = half a step of the type):

* norm + rotation: fp32 inside, so a value a cos - b sin is off by a few units of 2^-24 of |a| + |b| from the
  products, by the norm's own relative error (a sum of at most 256 squares in a tree, a square root and a
  division: below 12 units, half of the sum's counting) and by the final rounding:
  2^-20 (|a| + |b|) + u |y|.
* attention, bf16: the weights are rounded to bf16 (u = 2^-8 of each, so u times the weighted mean of |v|, in the
  numerator, and u |o| at most in the row sum where it adds up the rounded weights), the output once more (u |o|).
  The exponentials are off by at most 7.5e-5 relative, the scores by fp32 accumulation of D products, below
  D 2^-24 |q| |k| scale < 1e-4 here: together below 4e-4, numerator and row sum, < 2^-10 of the mean of |v|.
* attention, fp32: scores off by (D + 4) 2^-24 |q| |k| scale, exp2f and its argument by 4 units of the argument's
  size, sums over n keys by n 2^-24 at most: 2^-24 (2 n + 2 (D + 8) max|q||k| scale + 32) of the mean of |v|.
* LSE: the log of a row sum with the relative errors above; u = 2^-8 when the rounded weights are added up, else 4e-4.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import sequence_parallelism_st_b200 as st

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().double().numpy()


def rand(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def within(got, ref, tol, what):
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{what}: {np.count_nonzero(~np.isfinite(g))} values not finite"
    over = np.abs(g - ref) - tol
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what}: {np.count_nonzero(over > 0)} values off, worst at {at}: {g[at]} for {ref[at]} +- {np.broadcast_to(tol, ref.shape)[at]}"


# ---------------------------------------------------------------- norm and rotation
def check_qk(got, x, gamma, eps, table, pos, pairing, what):
    ref = oracle.qk_norm_rope(x, gamma, eps, table, pos, pairing)
    y = np.abs(oracle.qk_norm_rope(x, gamma, eps))
    D = y.shape[-1]
    pair = y + (y.reshape(*y.shape[:-1], D // 2, 2)[..., ::-1].reshape(y.shape) if pairing == "interleaved"
                else np.roll(y, D // 2, -1))
    within(got, ref, 2.0 ** -20 * pair + U[got.dtype] * np.abs(ref) + 1e-30, what)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("n,hq,hk,D", [(1, 16, 16, 72), (5, 1, 3, 8), (33, 24, 8, 128), (7, 5, 5, 256), (130, 2, 1, 32),
                                       (64, 7, 9, 80), (3, 3, 40, 96), (19, 16, 2, 64), (4, 2, 2, 136)])
def test_qk_norm_rope(dtype, pairing, n, hq, hk, D):
    q, k = rand(1, n, hq, D, dtype=dtype), rand(2, n, hk, D, dtype=dtype, scale=30.0)
    gq, gk = rand(3, D, dtype=F32) + 1, rand(4, D, dtype=F32)
    period = max(1, n // 3)
    table = st.st_rope_table(period, D)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    st.st_qk_norm_rope(q, k, qo, ko, gq, gk, 1e-6, rope_table=table, pos_period=period, pairing=pairing)
    pos = np.arange(n) % period
    check_qk(qo, q, gq, 1e-6, table, pos, pairing, "q")
    check_qk(ko, k, gk, 1e-6, table, pos, pairing, "k")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_qk_positions_fused_in_place(dtype):
    """Positions in and outside the table, Q and K as columns of one projection, in place: V's columns stay."""
    n, hq, hk, D = 50, 6, 2, 72
    x = rand(5, n, hq + 2 * hk, D, dtype=dtype)
    before = x.clone()
    table = st.st_rope_table(20, D)
    pos = torch.randint(-3, 24, (n,), generator=torch.Generator().manual_seed(6)).int()
    pos[:4] = torch.tensor([-2**31, 2**31 - 1, 19, 20])
    st.st_qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], eps=1e-5, rope_table=table, positions=pos.cuda(), pairing="halves")
    check_qk(x[:, :hq], before[:, :hq], None, 1e-5, table, pos.numpy(), "halves", "q")
    check_qk(x[:, hq:hq + hk], before[:, hq:hq + hk], None, 1e-5, table, pos.numpy(), "halves", "k")
    assert torch.equal(x[:, hq + hk:], before[:, hq + hk:])


def test_qk_one_tensor_no_rotation_zero_rows():
    """K of the text states alone; a row of zeros stays zero (eps), with eps = 0 it is NaN as the formula's."""
    k = rand(7, 2, 9, 4, 72)
    k[0, 3] = 0
    out = torch.full_like(k, 7.0)
    st.st_qk_norm_rope(None, k, None, out, k_gamma=torch.full((72,), 2.0, device="cuda"))
    check_qk(out.flatten(0, 1), k.flatten(0, 1), torch.full((72,), 2.0), 1e-6, None, None, "interleaved", "k")
    st.st_qk_norm_rope(k, None, out, eps=0.0)
    assert out[0, 3].isnan().all() and not out[1].isnan().any()


# ---------------------------------------------------------------- attention
def check_attn(q, segments, o, lse, scale=None, what=""):
    ref, rlse, mag = oracle.conditioned(q, segments, scale)
    sc = scale or 1 / math.sqrt(q.shape[-1])
    n = max(sum(s[0].shape[0] for s in c) for c in zip(*[[seg[b // (q.shape[0] // len(seg))] for b in range(q.shape[0])]
                                                      for seg in segments]))
    if q.dtype == BF:
        tol = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 * np.abs(ref) if o.dtype == BF else 0)
        ltol = 2.0 ** -8 + 4e-4
    else:
        kmax = max([float(s[0].double().norm(dim=-1).max()) if s[0].numel() else 0.0 for seg in segments for s in seg])
        smax = float(q.double().norm(dim=-1).max()) * kmax * sc
        rel = 2.0 ** -24 * (2 * n + 2 * (q.shape[-1] + 8) * smax + 32)
        tol, ltol = rel * mag + 2.0 ** -24 * np.abs(ref), rel + 2.0 ** -22 * (1 + smax)
    within(o, ref, tol + 1e-30, what + " o")
    if lse is not None:
        g = f64(lse)
        fin = np.isfinite(rlse)
        assert np.array_equal(g[~fin], rlse[~fin]), what + " lse of rows without keys"
        assert np.abs(g[fin] - rlse[fin]).max(initial=0.0) <= ltol, what + " lse"


def sets_of(k, v, length=None, offsets=None, mask=None, most=None):
    out = []
    if offsets is not None:
        off = offsets.cpu().tolist()
        for a, z in zip(off, off[1:]):
            out.append((k[a:z][:most], v[a:z][:most]))
        return out
    for i in range(k.shape[0]):
        n = k.shape[1] if length is None else int(length[i])
        ki, vi = k[i, :n], v[i, :n]
        if mask is not None:
            at = mask[i, :n].bool().nonzero().flatten()
            ki, vi = ki[at], vi[at]
        out.append((ki, vi))
    return out


def workspace(n):
    # poisoned: nothing in it may be taken for a result
    return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")


def run_cross(q, k, v, ws=True, o_fp32=0, scale=0.0, **kw):
    o = torch.full(q.shape, float("nan"), dtype=F32 if o_fp32 else q.dtype, device="cuda")
    lse = torch.full((q.shape[0], q.shape[1], q.shape[3], q.shape[2]), float("nan"), device="cuda")
    n = st.st_attn_cross_workspace_bytes(q, k, **kw, o_fp32=o_fp32)
    st.st_attn_cross(q, k, v, o, lse, workspace=workspace(n) if ws else None, o_fp32=o_fp32, scale=scale, **kw)
    assert st.st_check_device_status() == st.ST_OK
    return o, lse, n


HEAD_DIMS = [32, 64, 72, 80, 96, 128]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("B,T,S,H,L", [(1, 1, 1, 1, 1), (1, 2, 129, 2, 65), (2, 3, 37, 3, 300), (1, 1, 700, 1, 128)])
def test_cross(dtype, D, B, T, S, H, L):
    q, k, v = rand(10, B, T, S, H, D, dtype=dtype), rand(11, B, L, H, D, dtype=dtype), rand(12, B, L, H, D, dtype=dtype)
    o, lse, _ = run_cross(q, k, v)
    check_attn(q, [sets_of(k, v)], o, lse, what=f"cross D{D}")


@pytest.mark.parametrize("D", [30, 8, 1, 127])
def test_cross_fp32_other_head_dims(D):
    q, k, v = rand(13, 2, 1, 70, 2, D, dtype=F32), rand(14, 2, 66, 2, D, dtype=F32), rand(15, 2, 66, 2, D, dtype=F32)
    o, lse, _ = run_cross(q, k, v)
    check_attn(q, [sets_of(k, v)], o, lse, what=f"cross D{D}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [1, 5, 200])
@pytest.mark.parametrize("H,Hkv", [(6, 2), (8, 8), (5, 1), (12, 4)])
def test_cross_grouped_heads(dtype, S, H, Hkv):
    q, k, v = rand(16, 2, 2, S, H, 72, dtype=dtype), rand(17, 2, 90, Hkv, 72, dtype=dtype), rand(18, 2, 90, Hkv, 72, dtype=dtype)
    o, lse, _ = run_cross(q, k, v)
    check_attn(q, [sets_of(k, v)], o, lse, what="grouped")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [72, 128])
@pytest.mark.parametrize("S", [3, 300])
def test_cross_lengths_mask_packed_with_garbage(dtype, D, S):
    """Sets of 0, 1, part-tile, whole-tile and whole lengths; what does not count holds NaN and infinities."""
    L, H = 200, 2
    lens = torch.tensor([0, 1, 64, 65, 128, 200, 199, 63], dtype=torch.int32)
    n = len(lens)
    q = rand(20, n, 1, S, H, D, dtype=dtype)
    k, v = rand(21, n, L, H, D, dtype=dtype), rand(22, n, L, H, D, dtype=dtype)
    sets = sets_of(k, v, lens)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda", dtype=dtype)
    for i, m in enumerate(lens.tolist()):
        k[i, m:] = bad[i % 3]
        v[i, m:] = bad[(i + 1) % 3]
    o, lse, _ = run_cross(q, k, v, kv_len=lens.cuda())
    check_attn(q, [sets], o, lse, what="lengths")
    # the same through a mask
    mask = (torch.arange(L) < lens[:, None]).to(torch.uint8).cuda() * 3
    o2, lse2, _ = run_cross(q, k, v, kv_mask=mask)
    check_attn(q, [sets], o2, lse2, what="mask of lengths")
    # holes, whole tiles masked, a set with nothing left, and a length on top
    keep = torch.rand(n, L, generator=torch.Generator().manual_seed(23)) < 0.6
    keep[1, :] = False
    keep[2, :130] = False
    keep[3, 64:128] = False
    k, v = rand(24, n, L, H, D, dtype=dtype), rand(25, n, L, H, D, dtype=dtype)
    sets = sets_of(k, v, lens, mask=keep)
    k[~keep], v[~keep] = bad[0], bad[1]
    o, lse, _ = run_cross(q, k, v, kv_mask=keep.cuda(), kv_len=lens.cuda())
    check_attn(q, [sets], o, lse, what="mask and lengths")
    # packed, one sequence behind another, rows before, between and after them poisoned; some longer than max_len
    off = torch.zeros(n + 1, dtype=torch.int32)
    off[1:] = lens.cumsum(0)
    off += 3
    rows = int(off[-1]) + 40
    k, v = rand(26, rows, H, D, dtype=dtype), rand(27, rows, H, D, dtype=dtype)
    for x in (k, v):
        x[:3], x[int(off[-1]):] = bad[0], bad[1]
    o, lse, _ = run_cross(q, k, v, kv_offsets=off.cuda(), max_len=150)
    check_attn(q, [sets_of(k, v, offsets=off, most=150)], o, lse, what="packed")


def test_cross_lengths_and_offsets_out_of_range_are_clamped():
    q, k, v = rand(30, 3, 1, 20, 2, 72), rand(31, 3, 70, 2, 72), rand(32, 3, 70, 2, 72)
    o, lse, _ = run_cross(q, k, v, kv_len=torch.tensor([-5, 1000, 70], dtype=torch.int32).cuda())
    check_attn(q, [sets_of(k, v, torch.tensor([0, 70, 70]))], o, lse, what="lengths")
    kp, vp = k.flatten(0, 1), v.flatten(0, 1)
    o, lse, _ = run_cross(q, kp, vp, kv_offsets=torch.tensor([-7, 50, 20, 9999], dtype=torch.int32).cuda())
    sets = [(kp[:50], vp[:50]), (kp[:0], vp[:0]), (kp[20:], vp[20:])]
    check_attn(q, [sets], o, lse, what="offsets")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hkv,D,S,L", [(4, 4, 72, 1, 3000), (6, 2, 128, 1, 2000), (2, 2, 128, 70, 1500), (3, 1, 32, 5, 700)])
def test_cross_split(dtype, H, Hkv, D, S, L):
    """Few queries over many keys: the keys are split (a workspace is asked for) and combined; without one they are not."""
    lens = torch.tensor([L, 17, 0], dtype=torch.int32)
    q, k, v = rand(33, 3, 1, S, H, D, dtype=dtype), rand(34, 3, L, Hkv, D, dtype=dtype), rand(35, 3, L, Hkv, D, dtype=dtype)
    o, lse, n = run_cross(q, k, v, kv_len=lens.cuda())
    assert n > 0
    check_attn(q, [sets_of(k, v, lens)], o, lse, what="split")
    o, lse, _ = run_cross(q, k, v, ws=False, kv_len=lens.cuda())
    check_attn(q, [sets_of(k, v, lens)], o, lse, what="not split")
    o, lse, _ = run_cross(q, k, v, kv_len=lens.cuda(), o_fp32=1)
    check_attn(q, [sets_of(k, v, lens)], o, lse, what="split, fp32")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_cross_shared_states(dtype):
    """Sets shared by batches: whole runs of rows when they follow one another, batch by batch when they do not."""
    k, v = rand(36, 2, 130, 2, 72, dtype=dtype), rand(37, 2, 130, 2, 72, dtype=dtype)
    lens = torch.tensor([130, 40], dtype=torch.int32)
    q = rand(38, 6, 3, 50, 2, 72, dtype=dtype)
    o, lse, _ = run_cross(q, k, v, kv_len=lens.cuda())
    check_attn(q, [sets_of(k, v, lens)], o, lse, what="shared")
    wide = rand(39, 6, 3, 55, 2, 72, dtype=dtype)
    q = wide[:, :, :50]
    out = torch.zeros_like(wide)
    st.st_attn_cross(q, k, v, out[:, :, :50], kv_len=lens.cuda())
    check_attn(q, [sets_of(k, v, lens)], out[:, :, :50], None, what="strided")
    assert not out[:, :, 50:].any()                    # rows beside the queries stay as they were


@pytest.mark.parametrize("dtype", [BF, F32])
def test_cross_frame_blocks_and_scale(dtype):
    """Frames at a two-level stride (the sliced layouts), K and V as halves of one projection, another scale."""
    B, T, S, H, D = 2, 4, 40, 2, 72
    C = H * D
    big = rand(40, 2, B, 2, S + 3, C, dtype=dtype)     # [frame block, batch, frame in block, token, C]
    o = torch.zeros_like(big)
    kv = rand(41, B, 33, 2, H, D, dtype=dtype)
    k, v = kv[:, :, 0], kv[:, :, 1]
    sf, sb_ = (S + 3) * C, 2 * (S + 3) * C
    desc = st.make_desc(B, T, S, H, D, st._dtype_code(big), scale=0.5, stride_s=C, stride_t=sf, t_block=2,
                        stride_tb=B * sb_, stride_b=sb_)
    logical = big[:, :, :, :S].permute(1, 0, 2, 3, 4).reshape(B, T, S, H, D)
    lse = torch.zeros(B, T, H, S, device="cuda")
    if dtype == BF:                                    # the tensor maps need batches at whole frame blocks
        with pytest.raises(st.StattnError) as e:
            st.st_attn_cross(big, k, v, o, lse, desc=desc)
        assert e.value.code == st.ST_ERR_UNSUPPORTED
    big2 = big.permute(1, 0, 2, 3, 4).contiguous()     # [batch, frame block, frame in block, token, C]
    o2 = torch.zeros_like(big2)
    desc = st.make_desc(B, T, S, H, D, st._dtype_code(big), scale=0.5, stride_s=C, stride_t=sf, t_block=2,
                        stride_tb=2 * sf, stride_b=4 * sf)
    st.st_attn_cross(big2, k, v, o2, lse, desc=desc)
    check_attn(logical, [sets_of(k, v)], o2[:, :, :, :S].reshape(B, T, S, H, D), lse, scale=0.5, what="blocks")
    assert not o2[:, :, :, S:].any()


def run_prefix(q, kp, vp, k, v, ws=True, o_fp32=0, **kw):
    o = torch.full(q.shape, float("nan"), dtype=F32 if o_fp32 else q.dtype, device="cuda")
    lse = torch.full((q.shape[0], q.shape[1], q.shape[3], q.shape[2]), float("nan"), device="cuda")
    n = st.st_attn_prefix_workspace_bytes(q, kp, k, **kw, o_fp32=o_fp32)
    st.st_attn_prefix(q, kp, vp, k, v, o, lse, workspace=workspace(n) if ws else None, o_fp32=o_fp32, **kw)
    assert st.st_check_device_status() == st.ST_OK
    return o, lse, n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", HEAD_DIMS)
@pytest.mark.parametrize("B,sets,T,S,H,Hkv,Lp,L", [(2, 2, 1, 150, 2, 2, 70, 150), (4, 1, 1, 20, 2, 1, 100, 20),
                                                   (6, 2, 1, 1, 4, 2, 300, 9), (3, 1, 2, 3, 2, 2, 64, 40)])
def test_prefix(dtype, D, B, sets, T, S, H, Hkv, Lp, L):
    q = rand(50, B, T, S, H, D, dtype=dtype)
    kp, vp = rand(51, sets, Lp, Hkv, D, dtype=dtype), rand(52, sets, Lp, Hkv, D, dtype=dtype)
    k, v = rand(53, B, L, Hkv, D, dtype=dtype), rand(54, B, L, Hkv, D, dtype=dtype)
    for ws in (True, False):
        o, lse, _ = run_prefix(q, kp, vp, k, v, ws=ws)
        check_attn(q, [sets_of(kp, vp), sets_of(k, v)], o, lse, what=f"prefix ws={ws}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [1, 2, 170])
def test_prefix_ragged_and_masked(dtype, S):
    """Lengths on both sides (0 and whole), masks on both sides, poisoned rows; empty prefix and own keys together."""
    B, sets, H, Hkv, D, Lp, L = 6, 3, 4, 2, 72, 140, 70
    q = rand(60, B, 1, S, H, D, dtype=dtype)
    kp, vp = rand(61, sets, Lp, Hkv, D, dtype=dtype), rand(62, sets, Lp, Hkv, D, dtype=dtype)
    k, v = rand(63, B, L, Hkv, D, dtype=dtype), rand(64, B, L, Hkv, D, dtype=dtype)
    pl, ol = torch.tensor([140, 0, 65], dtype=torch.int32), torch.tensor([70, 0, 0, 1, 33, 64], dtype=torch.int32)
    pm = torch.rand(sets, Lp, generator=torch.Generator().manual_seed(65)) < 0.5
    om = torch.rand(B, L, generator=torch.Generator().manual_seed(66)) < 0.5
    om[4] = False
    segs = [sets_of(kp, vp, pl, mask=pm), sets_of(k, v, ol, mask=om)]
    pdead, odead = ~pm | (torch.arange(Lp) >= pl[:, None]), ~om | (torch.arange(L) >= ol[:, None])
    kp[pdead], vp[pdead], k[odead], v[odead] = float("nan"), float("inf"), float("-inf"), float("nan")
    for ws in (True, False):
        o, lse, _ = run_prefix(q, kp, vp, k, v, ws=ws, prefix_len=pl.cuda(), kv_len=ol.cuda(), prefix_mask=pm.cuda(),
                               kv_mask=om.cuda())
        check_attn(q, segs, o, lse, what=f"ragged ws={ws}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S", [1, 140])
def test_prefix_packed_rows_and_no_own_keys(dtype, S):
    B, H, D = 4, 2, 128
    q = rand(70, B, 1, S, H, D, dtype=dtype)
    off = torch.tensor([2, 77, 77, 78, 200], dtype=torch.int32)
    kp, vp = rand(71, 1, 90, H, D, dtype=dtype), rand(72, 1, 90, H, D, dtype=dtype)
    k, v = rand(73, 210, H, D, dtype=dtype), rand(74, 210, H, D, dtype=dtype)
    k[200:], v[200:] = float("nan"), float("nan")
    o, lse, _ = run_prefix(q, kp, vp, k, v, kv_offsets=off.cuda(), max_len=123)
    check_attn(q, [sets_of(kp, vp), sets_of(k, v, offsets=off)], o, lse, what="packed own")
    e = torch.zeros(B, 0, H, D, dtype=dtype, device="cuda")
    o, lse, _ = run_prefix(q, kp, vp, e, e)
    check_attn(q, [sets_of(kp, vp)], o, lse, what="no own keys")
    o, lse, _ = run_cross(q, e, e)
    assert not o.any() and (lse == -float("inf")).all()


def test_large_scores_and_late_maximum():
    """Scores that grow along the keys by far more than 2^8: the running maximum is raised in almost every step."""
    B, S, H, D, L = 1, 260, 2, 72, 640
    q = rand(80, B, 1, S, H, D)
    k, v = rand(81, B, L, H, D), rand(82, B, L, H, D)
    k = (k.float() * torch.linspace(0.2, 14, L, device="cuda")[None, :, None, None]).bfloat16()
    o, lse, _ = run_cross(q, k, v)
    ref, rlse, mag = oracle.conditioned(q, [sets_of(k, v)])
    # scores reach |q||k| scale ~ 100: fp32 accumulation is off by up to 80 * 2^-24 * 100 = 5e-4 relative there
    within(o, ref, (2.0 ** -8 + 2.0 ** -9) * mag + 2 * 2.0 ** -8 * np.abs(ref), "late maximum")
    assert np.abs(f64(lse) - rlse).max() <= 2.0 ** -8 + 1e-3


def test_partial_merges_with_the_framework():
    """An fp32 partial of the condition tokens, then st_attn_spatial_merge over the frame's own keys, is st_attn_prefix."""
    B, S, H, D, Lp = 2, 192, 2, 72, 100
    q, k, v = rand(90, B, 1, S, H, D), rand(91, B, 1, S, H, D), rand(92, B, 1, S, H, D)
    kp, vp = rand(93, B, Lp, H, D), rand(94, B, Lp, H, D)
    op, lp, _ = run_cross(q, kp, vp, o_fp32=1)
    o = torch.empty_like(q)
    st.st_attn_spatial_merge(q, k, v, op, lp, o)
    segs = [sets_of(kp, vp), sets_of(k[:, 0], v[:, 0])]
    ref, _, mag = oracle.conditioned(q, segs)
    within(o, ref, (2.0 ** -7 + 2.0 ** -9) * mag + 2.0 ** -7 * np.abs(ref), "merged")
    o2, _, _ = run_prefix(q, kp, vp, k[:, 0], v[:, 0])
    check_attn(q, segs, o2, None, what="prefix")


def conditioned_block(q, k, v, kt, vt, kp, vp, gq, gk, table, lens, out, ws):
    """One block's conditioning: norms and rotation, self-attention behind the prefix, cross attention to the text."""
    qn, kn = torch.empty_like(q), torch.empty_like(k)
    st.st_qk_norm_rope(q, k, qn, kn, gq, gk, rope_table=table, pos_period=q.shape[2])
    st.st_attn_prefix(qn, kp, vp, kn[:, 0], v[:, 0], out[0], workspace=ws)
    ktn = torch.empty_like(kt)
    st.st_qk_norm_rope(None, kt, None, ktn, k_gamma=gk)
    st.st_attn_cross(out[0], ktn, vt, out[1], kv_len=lens)


def test_operators_together_eager_captured_and_on_two_streams():
    """The operators as a block uses them, against the oracle; replayed from a graph with other inputs; two at once."""
    B, S, H, D, Lp, Lt = 2, 200, 2, 72, 96, 50
    def inputs(seed):
        x = [rand(seed + i, B, 1, S, H, D) for i in range(3)]
        x += [rand(seed + 3, B, Lt, H, D), rand(seed + 4, B, Lt, H, D), rand(seed + 5, 1, Lp, H, D), rand(seed + 6, 1, Lp, H, D)]
        return x + [rand(seed + 7, D, dtype=F32) + 1, rand(seed + 8, D, dtype=F32) + 1]
    table = st.st_rope_table(S, D)
    lens = torch.tensor([50, 7], dtype=torch.int32).cuda()
    def expect(x):
        q, k, v, kt, vt, kp, vp, gq, gk = x
        pos = np.arange(S).repeat(1)
        norm = lambda t, g: torch.from_numpy(np.stack([oracle.qk_norm_rope(t[b, 0], g, 1e-6, table, pos) for b in range(B)])[:, None])
        o1, _, m1 = oracle.conditioned(norm(q, gq), [sets_of(kp, vp), sets_of(norm(k, gk)[:, 0], v[:, 0].cpu())])
        return o1, m1
    def new_out():
        return [torch.zeros(B, 1, S, H, D, dtype=BF, device="cuda") for _ in range(2)]
    def check(x, out):
        o1, m1 = expect(x)
        # Q and K rounded to bf16 (2^-8 each) move a score by up to 2 * 2^-8 |s|, |s| <= |q||k| scale of normed heads
        smax = float((x[7].abs().max() * x[8].abs().max()) * math.sqrt(D))
        within(out[0], o1, (2.0 ** -7 * min(smax, 8.0) + 2.0 ** -7) * m1 + 2.0 ** -7 * np.abs(o1), "prefix")
        kt = torch.empty_like(x[3])
        st.st_qk_norm_rope(None, x[3], None, kt, k_gamma=x[8])
        check_attn(out[0], [sets_of(kt, x[4], lens)], out[1], None, what="cross")
    a, b = inputs(100), inputs(200)
    ws = workspace(st.st_attn_prefix_workspace_bytes(a[0], a[5], a[1][:, 0]))
    oa, ob = new_out(), new_out()
    conditioned_block(*a, table, lens, oa, ws)
    check(a, oa)
    # captured, replayed with other inputs in the same buffers
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    static = [t.clone() for t in a]
    with torch.cuda.stream(s):
        conditioned_block(*static, table, lens, ob, ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            conditioned_block(*static, table, lens, ob, ws)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(oa, ob))
    for t, n in zip(static, b):
        t.copy_(n)
    g.replay()
    torch.cuda.synchronize()
    check(b, ob)
    # two streams at once, each with its own workspace: the bits of the calls alone
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs, spaces = [new_out(), new_out()], [ws, ws.clone()]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, o, w, sm in zip((a, b), outs, spaces, streams):
            with torch.cuda.stream(sm):
                conditioned_block(*x, table, lens, o, w)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs[0], oa)) and all(torch.equal(x, y) for x, y in zip(outs[1], ob))


def test_results_do_not_depend_on_the_budget_or_the_run():
    q, k, v = rand(110, 2, 2, 300, 3, 72), rand(111, 2, 150, 3, 72), rand(112, 2, 150, 3, 72)
    o, lse, _ = run_cross(q, k, v)
    for sms in (0, 1, 37):
        st.st_set_sm_budget(sms)
        try:
            o2, lse2, _ = run_cross(q, k, v)
        finally:
            st.st_set_sm_budget(0)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,hq,hk,D", [(5001, 20, 20, 64), (9000, 3, 0, 40), (2500, 16, 16, 72), (20000, 1, 1, 256)])
def test_qk_many_tokens(dtype, n, hq, hk, D):
    """Every warp walks several tasks: three and four groups of bf16, head dims with and without their own kernel."""
    q, k = rand(120, n, hq, D, dtype=dtype), rand(121, n, hk, D, dtype=dtype) if hk else None
    qo, ko = torch.empty_like(q), torch.empty_like(k) if hk else None
    table = st.st_rope_table(977, D)
    st.st_qk_norm_rope(q, k, qo, ko, rope_table=table, pos_period=977)
    pos = np.arange(n) % 977
    check_qk(qo, q, None, 1e-6, table, pos, "interleaved", "q")
    if hk:
        check_qk(ko, k, None, 1e-6, table, pos, "interleaved", "k")


def test_qk_offsets_beyond_32_bits():
    """Tokens 2^31 elements and more apart from the first, in place."""
    n, step, H, D = 70, 2 ** 25, 2, 72
    big = torch.empty(n * step, dtype=BF, device="cuda")
    x = big.as_strided((n, H, D), (step, D, 1))
    x.copy_(rand(122, n, H, D))
    before = x.clone()
    assert (n - 1) * step > 2 ** 31
    st.st_qk_norm_rope(x, None, eps=1e-5)
    check_qk(x, before, None, 1e-5, None, None, "interleaved", "q")


@pytest.mark.parametrize("budget", [1, 3])
@pytest.mark.parametrize("D", [32, 72, 96, 128])
@pytest.mark.parametrize("L,lens", [(100, [100, 0, 17, 100]), (250, [250, 130, 0, 0]), (700, [0, 700, 1, 333])])
def test_cross_many_items_per_block(budget, D, L, lens):
    """One block and three walk all items: keys that stay and keys that stream, sets without keys between others,
    items of one, two and three row tiles, frames of one stride and frames with a gap."""
    H, Hkv = 2, 1
    k, v = rand(130, 4, L, Hkv, D), rand(131, 4, L, Hkv, D)
    n = torch.tensor(lens, dtype=torch.int32)
    sets = sets_of(k, v, n)
    for i, m in enumerate(lens):
        k[i, m:], v[i, m:] = float("nan"), float("inf")
    for T, S, gap in ((1, 460, 0), (3, 140, 9)):
        q = rand(132, 4, T, S + gap, H, D)[:, :, :S]
        o = torch.zeros(4, T, S + gap, H, D, dtype=BF, device="cuda")
        lse = torch.full((4, T, H, S), float("nan"), device="cuda")
        st.st_set_sm_budget(budget)
        try:
            st.st_attn_cross(q, k, v, o[:, :, :S], lse, kv_len=n.cuda())
            assert st.st_check_device_status() == st.ST_OK
        finally:
            st.st_set_sm_budget(0)
        check_attn(q, [sets], o[:, :, :S], lse, what=f"T{T}")
        assert not o[:, :, S:].any()
        o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
        st.st_attn_cross(q, k, v, o2[:, :, :S], lse2, kv_len=n.cuda())
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_sets", [40, 70, 200])
@pytest.mark.parametrize("D,S", [(72, 1), (128, 1), (72, 150), (128, 150)])
def test_cross_many_sets(dtype, n_sets, D, S):
    """More sets than a block keeps ranges of, as lengths and packed."""
    L, H = 90, 1
    n = torch.randint(0, L + 1, (n_sets,), generator=torch.Generator().manual_seed(133)).int()
    n[:3] = torch.tensor([L, 0, 1])
    q = rand(134, n_sets, 1, S, H, D, dtype=dtype)
    k, v = rand(135, n_sets, L, H, D, dtype=dtype), rand(136, n_sets, L, H, D, dtype=dtype)
    o, lse, _ = run_cross(q, k, v, kv_len=n.cuda())
    check_attn(q, [sets_of(k, v, n)], o, lse, what="lengths")
    off = torch.zeros(n_sets + 1, dtype=torch.int32)
    off[1:] = n.cumsum(0)
    kp, vp = k.flatten(0, 1), v.flatten(0, 1)
    o, lse, _ = run_cross(q, kp, vp, kv_offsets=off.cuda(), max_len=L)
    check_attn(q, [sets_of(kp, vp, offsets=off)], o, lse, what="packed")


@pytest.mark.parametrize("budget", [1, 2])
@pytest.mark.parametrize("H,Hkv,D,S,L", [(3, 3, 72, 5, 2600), (4, 2, 128, 1, 2300), (2, 1, 64, 70, 1700), (2, 2, 96, 130, 1300)])
def test_cross_split_parts_on_few_blocks(budget, H, Hkv, D, S, L):
    """The parts of split keys one behind another on one block, some of them empty: the bits of the whole GPU's run."""
    lens = torch.tensor([L, 0, 300], dtype=torch.int32)
    q, k, v = rand(140, 3, 1, S, H, D), rand(141, 3, L, Hkv, D), rand(142, 3, L, Hkv, D)
    o, lse, n = run_cross(q, k, v, kv_len=lens.cuda())
    assert n > 0
    check_attn(q, [sets_of(k, v, lens)], o, lse, what="split")
    st.st_set_sm_budget(budget)
    try:
        o2, lse2, n2 = run_cross(q, k, v, kv_len=lens.cuda())
    finally:
        st.st_set_sm_budget(0)
    assert n2 == n and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,L", [(3, 300), (16, 200), (17, 200)])
def test_cross_cut_by_cost(B, L):
    """Many items of sets of very different lengths; one set more than the cut by cost takes."""
    H, D, S = 2, 72, 2000
    n = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(143)).int()
    n[0], n[1] = L, 0
    q, k, v = rand(144, B, 1, S, H, D), rand(145, B, L, H, D), rand(146, B, L, H, D)
    st.st_set_sm_budget(7)
    try:
        o, lse, _ = run_cross(q, k, v, kv_len=n.cuda())
    finally:
        st.st_set_sm_budget(0)
    check_attn(q, [sets_of(k, v, n)], o, lse, what="cut")


@pytest.mark.parametrize("S", [1, 90])
def test_cross_fp32_rows_off_16_bytes(S):
    """fp32 rows need 4-byte alignment only: queries, keys and values one element on, odd strides."""
    H, D, L = 2, 32, 600
    def off(seed, n):
        x = torch.empty(n * (H * D + 3) + 1, device="cuda")
        t = x[1:].as_strided((1, n, H, D), (n * (H * D + 3), H * D + 3, D, 1))
        t.copy_(rand(seed, 1, n, H, D, dtype=F32))
        return t
    q, k, v = off(150, S)[:, None], off(151, L), off(152, L)
    o = off(153, S)[:, None]
    n = st.st_attn_cross_workspace_bytes(q, k)
    st.st_attn_cross(q, k, v, o, workspace=workspace(n))
    check_attn(q, [sets_of(k, v)], o, None, what="off")
    st.st_attn_prefix(q, k[:, :70], v[:, :70], k[:, 70:], v[:, 70:], o)
    check_attn(q, [sets_of(k, v)], o, None, what="prefix off")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_cross_offsets_beyond_32_bits(dtype):
    """A cache whose rows lie 2^31 elements and more behind the first."""
    L, step, H, D = 600, 2 ** 22, 2, 72
    def cache(seed):
        big = torch.empty(L * step, dtype=dtype, device="cuda")
        t = big.as_strided((1, L, H, D), (L * step, step, D, 1))
        t.copy_(rand(seed, 1, L, H, D, dtype=dtype))
        return t
    k, v = cache(160), cache(161)
    q = rand(162, 1, 1, 3, H, D, dtype=dtype)
    o, lse, _ = run_cross(q, k, v)
    check_attn(q, [sets_of(k.contiguous(), v.contiguous())], o, lse, what="long cache")
    # own keys of samples that share a prefix, left to the combine kernel
    kp, vp = rand(163, 1, 50, H, D, dtype=dtype), rand(164, 1, 50, H, D, dtype=dtype)
    ko, vo = (x.view(1, L, H, D).as_strided((2, L // 2, H, D), (L // 2 * step, step, D, 1)) for x in (k, v))
    q = rand(165, 2, 1, 1, H, D, dtype=dtype)
    o, lse, _ = run_prefix(q, kp, vp, ko, vo)
    check_attn(q, [sets_of(kp, vp), sets_of(ko.contiguous(), vo.contiguous())], o, lse, what="own keys")


@pytest.mark.parametrize("D", [72, 128])
@pytest.mark.parametrize("B,S,H,Hkv,Lp,L", [(40, 1, 4, 2, 2000, 130), (5, 30, 2, 2, 1000, 30), (130, 1, 2, 2, 90, 17)])
def test_prefix_packed_samples(D, B, S, H, Hkv, Lp, L):
    """Samples packed over a long prefix (one tile and several), own keys of every length beside it."""
    n = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(170)).int()
    n[0], n[1] = L, 0
    q = rand(171, B, 1, S, H, D)
    kp, vp = rand(172, 1, Lp, Hkv, D), rand(173, 1, Lp, Hkv, D)
    k, v = rand(174, B, L, Hkv, D), rand(175, B, L, Hkv, D)
    segs = [sets_of(kp, vp), sets_of(k, v, n)]
    for i, m in enumerate(n.tolist()):
        k[i, m:], v[i, m:] = float("nan"), float("nan")
    o, lse, ws = run_prefix(q, kp, vp, k, v, kv_len=n.cuda())
    assert ws > 0
    check_attn(q, segs, o, lse, what="packed")
    st.st_set_sm_budget(2)
    try:
        o2, lse2, _ = run_prefix(q, kp, vp, k, v, kv_len=n.cuda())
    finally:
        st.st_set_sm_budget(0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,S", [(72, 400), (128, 400), (72, 1)])
def test_cross_masks_with_dead_tails(dtype, D, S):
    """Masks whose last key is anywhere from none to the end of 1,300, at the end of the looks of 256 among them."""
    last = [0, 1, 255, 256, 257, 276, 277, 1043, 1044, 1045, 1299, 1300]
    B, L, H = len(last), 1300, 1
    q, k, v = rand(180, B, 1, S, H, D, dtype=dtype), rand(181, B, L, H, D, dtype=dtype), rand(182, B, L, H, D, dtype=dtype)
    keep = torch.zeros(B, L, dtype=torch.bool)
    for i, n in enumerate(last):
        keep[i, max(0, n - 700):n:3] = True
        if n:
            keep[i, n - 1] = True
    sets = sets_of(k, v, mask=keep)
    k[~keep], v[~keep] = float("nan"), float("inf")
    o, lse, _ = run_cross(q, k, v, kv_mask=keep.cuda())
    check_attn(q, [sets], o, lse, what="tails")
