"""Backward passes at values where a formula that is right in exact numbers can go wrong in fp32.

Bounds are those of test_gpu_backward.py (its head derives them) unless a test says what comes on top."""

import math

import pytest
import torch

import block_sparse_self_b200 as vsa
from test_gpu_backward import (DEV, U, bucket_of, check, inputs, list_mask, order_of, random_lists, reference,
                               window_mask)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    vsa.device_status()


# --------------------------------------------------------------------------
# centered dQ
# --------------------------------------------------------------------------

@pytest.mark.parametrize("mode", ["list", "window"])
def test_center_of_a_vanishing_mass(mode):
    """Keys 1 and 2 hold the weight, key 4 has e^-86 of it and the rest nothing: the columns that the mean key is
    weighted by (every fourth) have a mass of 16 e^-86, and the row's sum of dX over it is past fp32."""
    S, D = 128, 64
    g0 = torch.Generator(device=DEV).manual_seed(41)
    q = torch.zeros(1, 1, S, D, device=DEV)
    k = torch.zeros(1, 1, S, D, device=DEV)
    q[..., 0] = 8.0
    k[0, 0, :, 0] = -200.0          # logits of -200 and, at keys 1, 2 and 4, 86, 86 and 0 (exact in bf16 and fp32)
    k[0, 0, 1:3, 0] = 86.0
    k[0, 0, 4, 0] = 0.0
    k[..., 1:] = torch.randn(1, 1, S, D - 1, generator=g0, device=DEV)
    v = 100 * torch.randn(1, 1, S, D, generator=g0, device=DEV)
    g = 1000 * torch.randn(1, 1, S, D, generator=g0, device=DEV)
    q, k, v, g = (x.bfloat16() for x in (q, k, v, g))
    if mode == "list":
        lists = (torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV))
        o, lse = vsa.block_sparse_attention(q, k, v, *lists, 128, return_lse=True)
        got = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, *lists, 128, grad_dtype=torch.float32)
    else:
        o, lse = vsa.window_attention(q, k, v, S, return_lse=True)
        got = vsa.window_attention_backward(g, q, k, v, o, lse, S, grad_dtype=torch.float32)
    ref = reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], torch.ones(S, S, dtype=torch.bool, device=DEV))
    # the sums that the center is meant to take off do leave the range of fp32 when divided by that mass
    mass = 16 * math.exp(-86)
    assert (ref["e_dX"].sum(1) / mass).max() > torch.finfo(torch.float32).max
    check([x[0, 0] for x in got], ref)


def check_centered(dq, q, k, v, g, see):
    """dq against what independent roundings add up to where they multiply k - c, c the mean of the keys a row sees:
    var dq_i = scale^2 (u^2/3 sum_j dX_ij^2 (k_j - c)^2 + var delta_i (sum_j P_ij (k_j - c))^2), the two terms of
    test_gpu_backward.py, and for the sums that are taken off n roundings to fp32 of size |c| |dX|.  Five times that;
    with c = 0 (keys 16 times as far from zero as from one another) it would be 16 times."""
    ref = reference(q, k, v, g, see)
    k64, n = k.double(), see.sum(1, keepdim=True)
    scale = 1 / math.sqrt(q.shape[1])
    c = see.double() @ k64 / n
    P = torch.exp((scale * q.double() @ k64.T).masked_fill(~see, -math.inf) - ref["lse"][:, None])
    dX2 = ref["dX"] ** 2
    spread = (dX2 @ k64 ** 2 - 2 * c * (dX2 @ k64) + c ** 2 * dX2.sum(1, keepdim=True)).clamp(min=0)
    h2 = U * U / 3
    var_o = h2 * (ref["o"] ** 2 + P ** 2 @ v.double() ** 2 - 2 * ref["o"] * (P ** 2 @ v.double())
                  + ref["o"] ** 2 * (P ** 2).sum(1, keepdim=True))
    var_delta = (g.double() ** 2 * var_o).sum(1, keepdim=True)
    var = scale ** 2 * (h2 * spread + var_delta * (P @ k64 - c) ** 2 + n * 2.0 ** -48 * c ** 2 * dX2.sum(1, keepdim=True))
    assert (dq.double() - ref["dq"]).norm() <= 5 * var.sum().sqrt()


def far_keys(H, S, D):
    q, k, v, g = inputs(1, H, S, D, seed=S + D)
    m = torch.randn(1, H, 1, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    return (q.float() / 16).bfloat16(), (k.float() + 16 * m).bfloat16(), v, g


@pytest.mark.parametrize("block,nb,D,longest", [(128, 20, 128, 12), (64, 30, 64, 14), (32, 60, 128, 40), (128, 9, 64, 9),
                                                (128, 8, 64, 3)])
def test_lists_gradients_of_keys_with_a_large_mean(block, nb, D, longest):
    """dq's errors multiply the keys' spread and not their mean, however many blocks are listed."""
    H = 2
    q, k, v, g = far_keys(H, block * nb, D)
    idx, cnt = random_lists(1, H, nb, longest, seed=nb)
    o, lse, o_lo = vsa.block_sparse_attention(q, k, v, idx, cnt, block, return_remainder=True)
    dq = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block, grad_dtype=torch.float32, o_lo=o_lo)[0]
    for h in range(H):
        check_centered(dq[0, h], q[0, h], k[0, h], v[0, h], g[0, h], list_mask(idx[0, h], cnt[0, h], block, block * nb))


def test_sliding_tile_gradients_of_keys_with_a_large_mean():
    grid, H, D = (4, 24, 24), 2, 64
    S = math.prod(grid)
    q, k, v, g = far_keys(H, S, D)
    tok = order_of(grid, (4, 8, 8), grid).to(DEV)
    idx, cnt, group = vsa.structured_block_list("sliding_tile", grid)
    assert group == 0 and int(cnt.max()) > 8
    at = torch.empty(S, dtype=torch.long, device=DEV)
    at[tok] = torch.arange(S, device=DEV)
    see = list_mask(idx, cnt, 128, S)[at][:, at]
    args = (grid, [(4, 8, 8)], None, idx, cnt)
    o, lse, o_lo = vsa.block_sparse_attention_tiled(q, k, v, *args, return_remainder=True)
    dq = vsa.block_sparse_attention_tiled_backward(g, q, k, v, o, lse, *args, grad_dtype=torch.float32, o_lo=o_lo)[0]
    for h in range(H):
        check_centered(dq[0, h], q[0, h], k[0, h], v[0, h], g[0, h], see)


@pytest.mark.parametrize("block", [32, 64, 128])
def test_the_room_of_a_list_changes_nothing(block):
    """The same lists in wider rows: the same bits, forward and backward."""
    nb, D = 12, 64
    q, k, v, g = inputs(1, 2, block * nb, D, seed=block)
    idx, cnt = random_lists(1, 2, nb, 4, seed=block)
    res = []
    for cap in (4, 8, 9, 12):
        wide = torch.full((1, 2, nb, cap), -1, dtype=torch.int32, device=DEV)
        wide[..., :4] = idx
        o, lse, o_lo = vsa.block_sparse_attention(q, k, v, wide, cnt, block, return_remainder=True)
        res.append((o, lse, o_lo, *vsa.block_sparse_attention_backward(g, q, k, v, o, lse, wide, cnt, block, o_lo=o_lo)))
    for other in res[1:]:
        for x, y in zip(res[0], other):
            assert torch.equal(x, y)


# --------------------------------------------------------------------------
# bias entries of any size
# --------------------------------------------------------------------------

def buckets_of(S, buckets, far):
    f = torch.tensor([bucket_of(d, buckets, far) for d in range(far + 1)], device=DEV)
    i = torch.arange(S, device=DEV)
    r = i[None, :] - i[:, None]
    return f[r.abs().clamp(max=far)] + (r > 0) * (buckets // 2)


def large_tables(low, table):
    """Heads whose rows, some or all, see nothing but entries of the size of `low` (negative)."""
    b = torch.randn(16, 5, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    b[:8, 0] = low                    # masked by sign, the own key too: the last row sees masked keys only
    b[:, 1] += low                    # every entry: a common shift changes nothing
    b[0, 2] = -low                    # the own key far above everything else
    b[:4, 3] = low                    # three levels, the own key on the lowest: rows with three kinds of best key
    b[4:8, 3] = low / 2
    b[9:, 4] = 3 * low                # two levels, and single entries below the own key's
    b[3, 4] = low
    return b.to(table)


@pytest.mark.parametrize("low,table", [(-1e4, torch.float32), (-1e7, torch.float32), (-1e8, torch.bfloat16),
                                       (-1e9, torch.float32), (-1e30, torch.float32), (-5e37, torch.bfloat16)])
@pytest.mark.parametrize("S,D,window,sink", [(300, 64, 120, 2), (200, 128, 200, 0), (130, 64, 1, 0)])
def test_bias_entries_of_any_size(S, D, window, sink, low, table):
    """The softmax does not depend on the size of entries that a row sees nothing beside.

    Rows below one or two gaps have logits of up to 2^13 in the kernels (log2 units): rounding half a unit in the last
    place, 2^-11, four times (the saved logarithm twice, on its way to log2 units, the logit) moves a probability by
    4 ln 2 2^-11 < 0.36 u on top of the (2 + 1/16) u of the bounds: times 1.2."""
    H, far = 5, 64
    q, k, v, g = inputs(1, H, S, D, seed=S + 7)
    bias = large_tables(low, table)
    o, lse, o_lo = vsa.window_attention(q, k, v, window, sink, bias=bias, max_distance=far, return_remainder=True)
    *grads, dbias = vsa.window_attention_backward(g, q, k, v, o, lse, window, sink, bias=bias, max_distance=far,
                                                  grad_dtype=torch.float32, o_lo=o_lo)
    assert lse.isfinite().all()
    bucket, see = buckets_of(S, 16, far), window_mask(S, window, sink)
    want, err = (torch.zeros(16, H, dtype=torch.float64, device=DEV) for _ in range(2))
    for h in range(H):
        b = bias[:, h].double()[bucket]
        b -= b.masked_fill(~see, -math.inf).amax(1, keepdim=True)   # 64 bits do not hold a logit beside 1e30 either
        ref = reference(q[0, h], k[0, h], v[0, h], g[0, h], see, None, b)
        for name in ("o", "dq", "dk", "dv", "dX"):
            ref["e_" + name] = 1.2 * ref["e_" + name]
        assert ((o[0, h].double() - ref["o"]).abs() <= ref["e_o"] + 1e-6).all(), h
        check([x[0, h] for x in grads], ref, what=f"head {h}")
        want[:, h].index_add_(0, bucket.view(-1), ref["dX"].view(-1))
        err[:, h].index_add_(0, bucket.view(-1), ref["e_dX"].view(-1))
    if table == torch.bfloat16:
        err += U * (want.abs() + err)
    assert ((dbias.double() - want).abs() <= err + 1e-6).all()


def test_large_entries_leave_the_others_alone():
    """A mask by a large entry gives the bits of a mask by -inf where every row has another key, lse included."""
    S, D, H, far = 300, 64, 2, 64
    q, k, v, g = inputs(1, H, S, D, seed=31)
    bias = torch.randn(16, H, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    res = []
    for low in (-math.inf, -1e9, -1e4, torch.finfo(torch.float32).min):
        b = bias.clone()
        b[8:, 0] = low
        b[3, 1] = low
        o, lse = vsa.window_attention(q, k, v, 120, 2, bias=b, max_distance=far, return_lse=True)
        res.append((o, lse, *vsa.window_attention_backward(g, q, k, v, o, lse, 120, 2, bias=b, max_distance=far)))
    for other in res[1:]:
        for x, y in zip(res[0], other):
            assert torch.equal(x, y)


# --------------------------------------------------------------------------
# entries that are not finite
# --------------------------------------------------------------------------

@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("S,window,sink", [(16, 16, 0), (200, 40, 0), (300, 40, 3), (517, 100, 0)])
def test_bias_entries_that_are_not_finite_stay_with_their_pairs(S, window, sink, bad):
    """A NaN (or +inf) entry reaches the rows that see its bucket, the keys that those rows see, and nothing else.
    (At S = 16 offset 16, the first of a bucket, is that of positions past the end alone.)"""
    D, far = 64, 64
    q, k, v, g = inputs(1, 1, S, D, seed=32)
    table = torch.randn(16, 1, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    table[2] = -1e9             # with a gap to close
    bucket, see = buckets_of(S, 16, far), window_mask(S, window, sink)
    tile = torch.arange(S, device=DEV) // 128
    meet = torch.zeros(int(tile[-1]) + 1, int(tile[-1]) + 1, dtype=torch.bool, device=DEV)
    i, j = see.nonzero(as_tuple=True)
    meet[tile[i], tile[j]] = True       # tiles of queries and keys that are computed together

    ref = reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], see, None, table[:, 0].double()[bucket])
    err_db = torch.zeros(16, dtype=torch.float64, device=DEV).index_add_(0, bucket.view(-1), ref["e_dX"].view(-1))
    want_db = torch.zeros(16, dtype=torch.float64, device=DEV).index_add_(0, bucket.view(-1), ref["dX"].view(-1))

    def close(x, name, rows):
        return ((x.double() - ref[name]).abs() <= ref["e_" + name] + 1e-5)[rows].all()

    for at in (15, 14, 9, 7, 6):
        b = table.clone()
        b[at] = bad
        o, lse = vsa.window_attention(q, k, v, window, sink, bias=b, max_distance=far, out_dtype=torch.float32,
                                      return_lse=True)
        *grads, db = vsa.window_attention_backward(g, q, k, v, o, lse, window, sink, bias=b, max_distance=far,
                                                   grad_dtype=torch.float32)
        o, dq, dk, dv = (x[0, 0] for x in (o, *grads))
        hit = ((bucket == at) & see).any(1)
        seen = (hit[:, None] & see).any(0)
        assert o[hit].isnan().all() and dq[hit].isnan().all() and dk[seen].isnan().all() and dv[seen].isnan().all()
        assert close(o, "o", ~hit) and close(dq, "dq", ~hit) and close(dv, "dv", ~seen)
        # a masked pair of a computed tile is zero times the lost row's delta
        near = torch.stack([hit[tile == t].any() for t in range(len(meet))])
        assert close(dk, "dk", ~(near[:, None] & meet).any(0)[tile])
        if not hit.any():
            assert ((db[:, 0].double() - want_db).abs() <= err_db + 1e-5).all() and not db[at].any()


# --------------------------------------------------------------------------
# lse
# --------------------------------------------------------------------------

@pytest.mark.parametrize("mode,block,nb,D", [("lists", 128, 6, 128), ("lists", 64, 9, 64), ("lists", 32, 14, 128),
                                             ("lists", 128, 1, 64), ("tiled", 128, 8, 64), ("tiled", 64, 12, 128),
                                             ("window", 128, 5, 128), ("bias", 128, 5, 64)])
def test_lse_is_that_of_unrounded_exponentials(mode, block, nb, D):
    """Rows that a few keys of a later block hold: the bf16 rounding of their exponentials must not reach lse.

    With logits up to x = scale sum |q_d k_d| the accumulation of a product is off by D 2^-24 x at most, a sum of
    S <= 1024 exponentials by 2^-14 of itself, 2^x by 2^-22 and the last roundings by 2^-24 (|lse| + |m|), all of it
    below 2^-11 here (x <= 40).  P then carries its own rounding alone: |err dv_j| <= (u + u/16) sum_i P_ij |g_i|."""
    H, S = 2, block * nb
    q, k, v, g = inputs(1, H, S, D, seed=50 + S + D)
    q = (2 * q.float()).bfloat16()
    see, bias, args, kw = torch.ones(S, S, dtype=torch.bool, device=DEV), None, (), {}
    if mode in ("window", "bias"):
        fwd, bwd, args = vsa.window_attention, vsa.window_attention_backward, (200, 9)
        see = window_mask(S, 200, 9)
        if mode == "bias":
            table = torch.randn(16, H, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
            kw, bias = dict(bias=table, max_distance=64), table.double()[buckets_of(S, 16, 64)]
    else:
        idx = torch.arange(nb, dtype=torch.int32, device=DEV).expand(nb, nb).contiguous()
        cnt = torch.full((nb,), nb, dtype=torch.int32, device=DEV)
        fwd, bwd, args = vsa.block_sparse_attention, vsa.block_sparse_attention_backward, (idx, cnt, block)
        if mode == "tiled":
            grid = (nb, 8, block // 8)
            fwd, bwd = vsa.block_sparse_attention_tiled, vsa.block_sparse_attention_tiled_backward
            args = (grid, [(1, 8, block // 8)], None, idx, cnt)
    o, lse = fwd(q, k, v, *args, out_dtype=torch.float32, return_lse=True, **kw)
    dv = bwd(g, q, k, v, o, lse, *args, grad_dtype=torch.float32, **kw)[2]
    for h in range(H):
        assert (q[0, h].abs().float() @ k[0, h].abs().float().T).max() / math.sqrt(D) <= 40
        ref = reference(q[0, h], k[0, h], v[0, h], g[0, h], see, None, None if bias is None else bias[:, :, h])
        assert (lse[0, h].double() - ref["lse"]).abs().max() <= 2.0 ** -11
        ref["e_dv"] = ref["e_dv"] * (1 + 1 / 16) / (2 + 1 / 16)
        check([dv[0, h]], ref, names=("dv",))


# --------------------------------------------------------------------------
# buckets
# --------------------------------------------------------------------------

@pytest.mark.parametrize("buckets,far,border", [(96, 4010233, 198349), (106, 8670623, 125033), (244, 13223778, 352201),
                                                (36, 6102237, 1372691), (32, 128, 64), (64, 4096, 512), (20, 2560, 320)])
def test_bucket_borders_next_to_whole_numbers(buckets, far, border):
    """Borders that lie within 10^-13 above a whole number (it is still in the lower bucket), and on one."""
    got = vsa.relative_position_buckets(buckets, far)
    for d in (border - 1, border, border + 1, border + 2):
        if d <= far:
            assert int(got[far - d]) == bucket_of(d, buckets, far)
            assert int(got[far + d]) == buckets // 2 + bucket_of(d, buckets, far)


# --------------------------------------------------------------------------
# joined parts
# --------------------------------------------------------------------------

@pytest.mark.parametrize("mode,block,nb,D", [("short lists", 128, 6, 64), ("short lists", 32, 14, 128),
                                             ("long lists", 32, 40, 64), ("long lists", 64, 24, 128),
                                             ("window and lists", 128, 5, 64)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_gradients_of_joined_parts(mode, block, nb, D, out):
    """A softmax over two sets of keys, each by a call of its own: every part's gradients from the joined o and lse.

    A part's sum of dX is no error.  Only where it is at most 2u sum_d |g_d o_d| = 2u G_i may it be taken for one; the
    bounds of dX grow by P_ij 2u G_i for that, and where dq is centered its own by scale 2u G_i max |k|.  Joining in
    fp32 adds nothing to the half step of a bf16 o that the bounds have."""
    H, S = 2, block * nb
    q, k, v, g = inputs(1, H, S, D, seed=60 + S + D)
    b = torch.arange(nb)
    if mode == "window and lists":      # the window reaches 30 positions, the lists two blocks on
        parts = [("window", (60, 0)), ("lists", [[(i + 2) % nb] for i in range(nb)])]
    else:
        n = 3 if mode == "short lists" else nb // 2
        parts = [("lists", [sorted((i * 5 + s + 2 * e) % nb for e in range(n)) for i in range(nb)]) for s in (0, 1)]
    see, res = torch.zeros(S, S, dtype=torch.bool, device=DEV), []
    for kind, what in parts:
        if kind == "window":
            fwd, bwd, args = vsa.window_attention, vsa.window_attention_backward, what
            mine = window_mask(S, *what)
        else:
            idx = torch.tensor(what, dtype=torch.int32, device=DEV)
            cnt = torch.full((nb,), idx.shape[1], dtype=torch.int32, device=DEV)
            fwd, bwd, args = vsa.block_sparse_attention, vsa.block_sparse_attention_backward, (idx, cnt, block)
            mine = list_mask(idx, cnt, block, S)
        assert not (see & mine).any()
        see |= mine
        res.append((*fwd(q, k, v, *args, out_dtype=torch.float32, return_lse=True), bwd, args))
    lse = torch.logaddexp(res[0][1], res[1][1])
    o = sum(x[0] * (x[1] - lse).exp()[..., None] for x in res).to(out)
    dq, dk, dv = (sum(x) for x in zip(*(bwd(g, q, k, v, o, lse, *args, grad_dtype=torch.float32)
                                        for _, _, bwd, args in res)))
    scale = 1 / math.sqrt(D)
    for h in range(H):
        ref = reference(q[0, h], k[0, h], v[0, h], g[0, h], see)
        q64, k64, v64, g64 = (x[0, h].double() for x in (q, k, v, g))
        P = torch.exp((scale * q64 @ k64.T).masked_fill(~see, -math.inf) - ref["lse"][:, None])
        G = 2 * U * (g64.abs() * ref["o"].abs()).sum(1, keepdim=True)
        extra = P * G
        bounds = dict(dq=ref["e_dq"] + scale * (extra @ k64.abs() + 2 * G * k64.abs().max()),
                      dk=ref["e_dk"] + scale * extra.T @ q64.abs(), dv=ref["e_dv"])
        for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
            off = (x[0, h].double() - ref[name]).abs()
            assert (off <= bounds[name] + 1e-5).all(), name
            assert off.norm() <= 0.02 * ref[name].norm(), name     # what is missing otherwise is of its own size


# --------------------------------------------------------------------------
# groups that are not a power of two and cross blocks; blocks of 32 and 64 under structured masks
# --------------------------------------------------------------------------

@pytest.mark.parametrize("block,nb,D,group", [(128, 4, 64, 96), (128, 5, 128, 100), (128, 3, 64, 200), (64, 7, 128, 48),
                                              (64, 6, 64, 130), (32, 13, 64, 24), (32, 9, 128, 37)])
def test_groups_that_cross_blocks(block, nb, D, group):
    """A row's group of keys lies in one listed block or in several; the last group is cut by the end."""
    H, S = 2, block * nb
    q, k, v, g = inputs(1, H, S, D, seed=S + group)
    i = torch.arange(nb)
    lo, hi = i * block // group * group // block, ((i * block + block - 1) // group * group + group - 1) // block
    lists = [list(range(int(a), min(int(b), nb - 1) + 1)) for a, b in zip(lo, hi)]
    lists[-1] = sorted({0, *lists[-1]})     # a block that none of its rows sees a key of
    cap = max(map(len, lists))
    idx = torch.tensor([x + [-1] * (cap - len(x)) for x in lists], dtype=torch.int32, device=DEV)
    cnt = torch.tensor([len(x) for x in lists], dtype=torch.int32, device=DEV)
    p = torch.arange(S, device=DEV) // group
    see = list_mask(idx, cnt, block, S) & (p[:, None] == p)
    assert (see == (p[:, None] == p)).all()
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, group, return_lse=True)
    got = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block, group, grad_dtype=torch.float32)
    for h in range(H):
        ref = reference(q[0, h], k[0, h], v[0, h], g[0, h], see)
        assert ((o[0, h].double() - ref["o"]).abs() <= ref["e_o"] + 1e-6).all()
        check([x[0, h] for x in got], ref, what=f"head {h}")


@pytest.mark.parametrize("kind,grid,block", [("spatial", (3, 8, 12), 32), ("temporal", (16, 4, 8), 64), ("temporal", (8, 4, 8), 32),
                                             ("spatial", (6, 4, 8), 64), ("temporal", (64, 2, 4), 32)])
def test_structured_masks_of_short_blocks(kind, grid, block):
    """The path of permuted tensors and groups, differentiated through."""
    D, H = 64, 2
    S = math.prod(grid)
    q, k, v, g = inputs(1, H, S, D, seed=S + block)
    plain = vsa.structured_attention(q, k, v, kind, grid, block)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = vsa.structured_attention(*leaves, kind, grid, block)
    assert (o - plain).abs().max() <= 4 * U * v.abs().max()     # another kernel's rounding
    got = torch.autograd.grad(o, leaves, g)
    i = torch.arange(S, device=DEV)
    label = i // (grid[1] * grid[2]) if kind == "spatial" else i % (grid[1] * grid[2])
    for h in range(H):
        check([x[0, h] for x in got], reference(q[0, h], k[0, h], v[0, h], g[0, h], label[:, None] == label))
