"""Backward passes of the attention calls, the relative position bias and the
transposed block lists against plain 64-bit computations.

Tolerances are worst cases, computed element by element from the 64-bit values
(u = 2^-8, half a step of bf16; the kernels round three things to it):

* P enters PV and dV rounded (u), and the forward row sum adds rounded P, so a
  probability recomputed from lse is off by at most u more; fp32 products and
  exponentials add less than u / 16 for the logits used here.
* the forward output is a sum of v_j with weights off by at most 2u, then
  rounded (u) when it is bf16: |err o_i| <= 2u sum_j P_ij |v_j| + u |o_i|;
  delta_i = g_i.o_i carries |g_i| times that.
* dX = P (g.v - delta) is rounded (u) on its way to dQ and dK.
So with W = 2u + u/16,
  |err dv_j| <= W sum_i P_ij |g_i|
  |err dX_ij| <= W |dX_ij| + P_ij |err delta_i| + c P_ij |g_i|.|v_j|
(c = 2^-16: fp32 accumulation over D <= 128 terms, both ways) and dq, dk, dbias
take the sums of that with |k|, |q| and 1.  bf16 gradients add u of the value.

The worst case leaves room for a small mistake, so each whole gradient is also
held to five times what independent roundings add up to (2-norm).  A rounding
has a variance of at most u^2/3 of the squared value, so
  var delta_i = u^2/3 sum_d g_id^2 (o_id^2 + sum_j P_ij^2 (v_jd - o_id)^2)
  var dX_ij = u^2/3 dX_ij^2 (its own) + P_ij^2 var delta_i, the latter one error
of a whole row; lse is one relative error of at most u per row, variance u^2/3:
  var dq_i = scale^2 (u^2/3 sum_j dX_ij^2 k_j^2 + var delta_i (sum_j P_ij k_j)^2) + u^2/3 dq_i^2
  var dk_j = scale^2 sum_i (2 u^2/3 dX_ij^2 + P_ij^2 var delta_i) q_i^2
  var dv_j = 2 u^2/3 sum_i P_ij^2 g_i^2
(A flat limit of 2u of the gradient's norm would be wrong: a row held by one of
two keys has a dX far below P |g| |o|, and delta's u |g| |o| stays.)
"""

import math

import pytest
import torch

import block_sparse_self_b200 as vsa

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
W = 2 * U + U / 16
C32 = 2.0 ** -16
DEV = "cuda"


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    vsa.device_status()


def order_of(grid, tile, pgrid):
    """Token at each position of the tile-contiguous order over the padded grid; -1 at padding."""
    p = torch.arange(math.prod(pgrid))
    t, h, w = p // (pgrid[1] * pgrid[2]), p // pgrid[2] % pgrid[1], p % pgrid[2]
    label = ((t // tile[0]) * (pgrid[1] // tile[1]) + h // tile[1]) * (pgrid[2] // tile[2]) + w // tile[2]
    tok = torch.where((t < grid[0]) & (h < grid[1]) & (w < grid[2]), (t * grid[1] + h) * grid[2] + w, -1)
    return tok[torch.argsort(label, stable=True)]


def random_lists(B, H, nb, longest, seed, shared=False):
    """Ascending lists of 1 to `longest` distinct blocks; the first query block lists as many as it may."""
    g = torch.Generator().manual_seed(seed)
    lead = () if shared else (B, H)
    longest = min(longest, nb)
    n = math.prod(lead) * nb
    keys = torch.rand(n, nb, generator=g).argsort(1)[:, :longest]
    cnt = torch.randint(1, longest + 1, (n,), generator=g)
    cnt[0] = longest
    idx = torch.full((n, longest), -1)
    for r in range(n):
        idx[r, :cnt[r]] = keys[r, :cnt[r]].sort().values
    return (idx.int().view(*lead, nb, longest).to(DEV).contiguous(), cnt.int().view(*lead, nb).to(DEV).contiguous())


def list_mask(idx, cnt, block, positions):
    """[positions, positions] visibility of one head's lists."""
    nb = positions // block
    m = torch.zeros(nb, nb, dtype=torch.bool)
    for i in range(nb):
        m[i, idx[i, :cnt[i]].long().cpu()] = True
    return m.repeat_interleave(block, 0).repeat_interleave(block, 1).to(DEV)


def inputs(B, H, S, D, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = [torch.randn(B, H, S, D, generator=g, device=DEV) for _ in range(4)]
    x[0] *= 1.5  # logits with a standard deviation of 1.5
    return [y.to(dtype) for y in x]


def reference(q, k, v, g, see, scale=None, bias=None):
    """One head in 64 bits: o, lse, dq, dk, dv, dX, and what each may be off by.  see [S, S] bool, bias [S, S]."""
    q, k, v, g = (x.double() for x in (q, k, v, g))
    scale = 1 / math.sqrt(q.shape[1]) if scale is None else scale
    x = scale * (q @ k.T) + (0 if bias is None else bias)
    x = x.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(x, 1)
    live = torch.isfinite(lse)
    P = torch.where(live[:, None], torch.exp(x - lse.masked_fill(~live, 0)[:, None]), 0.0)
    o = P @ v
    delta = (g * o).sum(1)
    dX = P * (g @ v.T - delta[:, None])
    h2 = U * U / 3
    var_o = h2 * (o ** 2 + P ** 2 @ v ** 2 - 2 * o * (P ** 2 @ v) + o ** 2 * (P ** 2).sum(1, keepdim=True))
    var_delta = (g ** 2 * var_o).sum(1, keepdim=True)
    s_dq = scale ** 2 * (h2 * dX ** 2 @ k ** 2 + var_delta * (P @ k) ** 2) + h2 * (scale * dX @ k) ** 2
    s_dk = scale ** 2 * (2 * h2 * dX ** 2 + P ** 2 * var_delta).T @ q ** 2
    s_dv = 2 * h2 * (P ** 2).T @ g ** 2
    err_o = 2 * U * (P @ v.abs()) + U * o.abs()
    err_delta = (g.abs() * err_o).sum(1)
    err_dX = W * dX.abs() + P * err_delta[:, None] + C32 * P * (g.abs() @ v.abs().T)
    return dict(o=o, lse=lse, dX=dX, dq=scale * dX @ k, dk=scale * dX.T @ q, dv=P.T @ g,
                e_o=err_o + U / 16 * (P @ v.abs()), e_dX=err_dX, e_dq=scale * err_dX @ k.abs(),
                e_dk=scale * err_dX.T @ q.abs(), e_dv=W * (P.T @ g.abs()), s_dq=s_dq, s_dk=s_dk, s_dv=s_dv)


def check(got, ref, names=("dq", "dk", "dv"), what=""):
    for x, name in zip(got, names):
        want, err = ref[name], ref["e_" + name]
        assert torch.isfinite(x).all(), f"{what} {name}"
        if x.dtype == torch.bfloat16:
            err = err + U * (want.abs() + err)
        off = (x.double() - want).abs() - err
        # fp32 sums of many terms
        off -= C32 * want.abs() + 1e-6
        assert off.max() <= 0, f"{what} {name}: {off.max():.3e} over the bound at {int(off.argmax())}"
        var = ref["s_" + name] + (U * U / 3 * want ** 2 if x.dtype == torch.bfloat16 else 0)
        far = (x.double() - want).norm() / (var.sum().sqrt() + C32 * want.norm() + 1e-6)
        assert far <= 5, f"{what} {name}: {far:.2f} times what independent roundings give"


# --------------------------------------------------------------------------
# transposed lists
# --------------------------------------------------------------------------

@pytest.mark.parametrize("B,H,nb,longest,shared", [
    (1, 1, 1, 1, False), (1, 2, 3, 2, False), (2, 3, 31, 7, False), (1, 2, 32, 32, False), (1, 1, 33, 5, True),
    (1, 3, 257, 40, False), (1, 1, 1100, 9, True), (1, 1, 8200, 3, True),
])
def test_transposed_lists(B, H, nb, longest, shared):
    idx, cnt = random_lists(B, H, nb, longest, seed=nb, shared=shared)
    off, rows = vsa.transpose_block_lists(idx, cnt)
    assert off.shape == cnt.shape[:-1] + (nb + 1,) and rows.shape == cnt.shape[:-1] + (nb * idx.shape[-1],)
    for i, c, o, r in zip(idx.reshape(-1, nb, idx.shape[-1]).tolist(), cnt.reshape(-1, nb).tolist(),
                          off.reshape(-1, nb + 1).tolist(), rows.reshape(-1, rows.shape[-1]).tolist()):
        who = [[] for _ in range(nb)]
        for q in range(nb):
            for key in i[q][:c[q]]:
                who[key].append(q)
        flat = [q for w in who for q in w]
        assert o == [0] + torch.tensor([len(w) for w in who]).cumsum(0).tolist()
        assert r == flat + [-1] * (len(r) - len(flat))


def test_transposed_lists_empty_and_invalid():
    # an empty list names nothing; a list out of range, out of order or too long names nothing and is reported
    idx = torch.tensor([[0, 2], [-1, -1], [1, 2]], dtype=torch.int32, device=DEV)
    off, rows = vsa.transpose_block_lists(idx, torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV))
    assert off.tolist() == [0, 1, 2, 3] and rows.tolist() == [0, 2, 0, -1, -1, -1]
    vsa.device_status()
    for bad, cnt in (([[0, 3], [0, 1], [1, 2]], [2, 2, 2]), ([[2, 1], [0, 1], [1, 2]], [2, 2, 2]),
                     ([[0, 1], [0, 1], [1, 2]], [3, 2, 2]), ([[1, 1], [0, 1], [1, 2]], [2, 2, 2])):
        off, rows = vsa.transpose_block_lists(torch.tensor(bad, dtype=torch.int32, device=DEV),
                                              torch.tensor(cnt, dtype=torch.int32, device=DEV))
        assert off.tolist() == [0, 1, 3, 4] and rows.tolist() == [1, 1, 2, 2, -1, -1]
        with pytest.raises(RuntimeError):
            vsa.device_status()


# --------------------------------------------------------------------------
# block lists in tile-contiguous order
# --------------------------------------------------------------------------

@pytest.mark.parametrize("block,nb,D,longest,shared,group,scale", [
    (128, 1, 64, 1, False, 0, None),        # one block
    (128, 5, 128, 1, False, 0, None),       # lists of one block: the forward pass's one-block kernel
    (128, 7, 64, 4, False, 0, None),
    (128, 6, 128, 6, False, 0, 0.2),
    (128, 4, 128, 3, True, 0, None),        # one list for every head
    (128, 3, 64, 1, True, 32, None),        # groups
    (64, 9, 128, 4, False, 0, None),        # an odd number of 64-token blocks per list
    (64, 5, 64, 5, False, 0, None),
    (32, 11, 64, 7, False, 0, None),
    (32, 6, 128, 3, False, 16, 0.1),
])
def test_block_sparse_backward(block, nb, D, longest, shared, group, scale):
    B, H = 2, 2
    S = block * nb
    q, k, v, g = inputs(B, H, S, D, seed=block + nb + D)
    idx, cnt = random_lists(B, H, nb, longest, seed=nb, shared=shared)
    if group:  # a row must see a key: groups reach inside the diagonal block
        idx = torch.arange(nb, dtype=torch.int32, device=DEV).view(nb, 1).contiguous()
        cnt = torch.ones(nb, dtype=torch.int32, device=DEV)
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, group, scale, return_lse=True)
    plain = vsa.block_sparse_attention(q, k, v, idx, cnt, block, group, scale)
    # 32- and 64-token blocks have a forward kernel of their own beside lse: o is then rounded differently
    assert torch.equal(o, plain) if block == 128 else (o - plain).abs().max() <= 4 * U * v.abs().max()
    args = (idx, cnt, block, group, scale)
    low = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, *args)
    full = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, *args, grad_dtype=torch.float32)
    again = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, *args, grad_dtype=torch.float32)
    for x, y, z in zip(low, full, again):
        assert torch.equal(y, z)                       # one order of every sum
        assert torch.equal(x, y.to(torch.bfloat16))    # rounded once
    p = torch.arange(S, device=DEV)
    for b in range(B):
        for h in range(H):
            see = list_mask(*((idx, cnt) if idx.dim() == 2 else (idx[b, h], cnt[b, h])), block, S)
            if group:
                see &= (p[:, None] // group) == (p[None, :] // group)
            ref = reference(q[b, h], k[b, h], v[b, h], g[b, h], see, scale)
            assert (lse[b, h].double() - ref["lse"]).abs().max() <= W
            check([x[b, h] for x in full], ref, what=f"head {b},{h}")
            check([x[b, h] for x in low], ref, what=f"head {b},{h}")


def test_block_sparse_backward_unlisted_keys_and_bad_lists():
    # keys that no list names get zeros; a query block with a bad list passes nothing on; the rest is unharmed
    B, H, nb, D, block = 1, 1, 4, 64, 128
    S = nb * block
    q, k, v, g = inputs(B, H, S, D, seed=5)
    idx = torch.tensor([[0, 1], [9, 1], [0, 1], [1, -1]], dtype=torch.int32, device=DEV).view(1, 1, nb, 2)
    cnt = torch.tensor([2, 2, 2, 1], dtype=torch.int32, device=DEV).view(1, 1, nb)
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, return_lse=True)
    with pytest.raises(RuntimeError):
        vsa.device_status()
    assert (lse[0, 0, block:2 * block] == -math.inf).all()
    dq, dk, dv = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block, grad_dtype=torch.float32)
    with pytest.raises(RuntimeError):
        vsa.device_status()
    see = torch.zeros(S, S, dtype=torch.bool, device=DEV)
    see[:block, :2 * block] = see[2 * block:3 * block, :2 * block] = see[3 * block:, block:2 * block] = True
    check([x[0, 0] for x in (dq, dk, dv)], reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], see))
    assert not dq[0, 0, block:2 * block].any() and not dk[0, 0, 2 * block:].any() and not dv[0, 0, 2 * block:].any()


def test_block_sparse_backward_rows_that_see_nothing():
    # groups of 32 that lie outside the listed block: those rows have no key, o = 0, and pass nothing on
    D, block, nb = 64, 128, 2
    S = nb * block
    q, k, v, g = inputs(1, 1, S, D, seed=8)
    idx = torch.tensor([[0], [0]], dtype=torch.int32, device=DEV)
    cnt = torch.ones(2, dtype=torch.int32, device=DEV)
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, 32, return_lse=True)
    with pytest.raises(RuntimeError):
        vsa.device_status()
    dq, dk, dv = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block, 32, grad_dtype=torch.float32)
    assert (lse[0, 0, block:] == -math.inf).all() and not o[0, 0, block:].any()
    assert not dq[0, 0, block:].any() and not dk[0, 0, block:].any() and not dv[0, 0, block:].any()
    p = torch.arange(S, device=DEV)
    see = ((p[:, None] // 32) == (p[None, :] // 32)) & (p[None, :] < block)
    check([x[0, 0] for x in (dq, dk, dv)], reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], see))


def test_values_of_unlisted_blocks_are_not_read():
    D, block, nb = 64, 128, 4
    q, k, v, g = inputs(1, 1, nb * block, D, seed=9)
    idx = torch.tensor([[0, 2], [0, 1], [1, 2], [0, 1]], dtype=torch.int32, device=DEV)
    cnt = torch.full((nb,), 2, dtype=torch.int32, device=DEV)
    out = []
    for bad in (False, True):
        if bad:
            k, v = k.clone(), v.clone()
            k[:, :, 3 * block:], v[:, :, 3 * block:] = math.nan, math.inf
        o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, return_lse=True)
        out.append(vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block))
    for x, y in zip(*out):
        assert torch.equal(x, y)


# --------------------------------------------------------------------------
# T-major tensors, a tiling per head
# --------------------------------------------------------------------------

@pytest.mark.parametrize("grid,tiles,D,longest,stride", [
    ((4, 8, 16), [(1, 8, 16), (2, 8, 8), (4, 4, 8)], 128, 3, 0),
    ((3, 9, 17), [(1, 8, 16), (2, 8, 8)], 64, 4, 0),            # padded on every axis
    ((5, 13, 20), [(4, 4, 8)], 128, 5, 0),
    ((4, 8, 16), [(4, 8, 8)], 64, 2, 0),                        # tiles of two blocks
    ((4, 8, 32), [(4, 1, 32)], 128, 2, 32),                     # strided groups: same (h, w)
    ((3, 9, 20), [(1, 4, 16), (1, 8, 8)], 128, 7, 0),           # 64-token tiles, padded
    ((4, 6, 12), [(2, 4, 4)], 64, 5, 0),                        # 32-token tiles, padded
])
def test_tiled_backward(grid, tiles, D, longest, stride):
    B, H = 1, 3
    S = math.prod(grid)
    pg = vsa.padded_grid(grid, tiles)
    positions, block = math.prod(pg), min(128, math.prod(tiles[0]))
    nb = positions // block
    q, k, v, g = inputs(B, H, S, D, seed=S)
    choice = (torch.arange(B * H) % len(tiles)).int().to(DEV)
    idx, cnt = random_lists(B, H, nb, longest, seed=S)
    # every list names block 0, which holds token 0: no row is without a key
    idx[..., 0] = 0
    orders = [order_of(grid, t, pg) for t in tiles]
    masks = []
    for h in range(H):
        tok = orders[int(choice[h])].to(DEV)
        see = list_mask(idx[0, h], cnt[0, h], block, positions)
        p = torch.arange(positions, device=DEV)
        if stride:
            see &= (p[:, None] - p[None, :]) % stride == 0
        at = torch.empty(S, dtype=torch.long, device=DEV)
        at[tok[tok >= 0]] = p[tok >= 0]   # position of each token
        masks.append(see[at][:, at])
    assert all(m.any(1).all() for m in masks)  # what the lists above are made for
    o, lse = vsa.block_sparse_attention_tiled(q, k, v, grid, tiles, choice, idx, cnt, group_stride=stride, return_lse=True)
    args = (grid, tiles, choice, idx, cnt)
    full = vsa.block_sparse_attention_tiled_backward(g, q, k, v, o, lse, *args, group_stride=stride,
                                                     grad_dtype=torch.float32)
    low = vsa.block_sparse_attention_tiled_backward(g, q, k, v, o, lse, *args, group_stride=stride)
    for x, y in zip(low, full):
        assert torch.equal(x, y.to(torch.bfloat16))
    for h in range(H):
        ref = reference(q[0, h], k[0, h], v[0, h], g[0, h], masks[h])
        assert (lse[0, h].double() - ref["lse"]).abs().max() <= W
        check([x[0, h] for x in full], ref, what=f"head {h}")


def test_tiled_backward_equals_permuted():
    grid, tiles, D, H = (4, 16, 16), [(1, 8, 16), (2, 8, 8), (4, 4, 8)], 128, 3
    q, k, v, g = inputs(1, H, math.prod(grid), D, seed=3)
    choice = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    idx, cnt = random_lists(1, H, 8, 5, seed=3)
    o, lse = vsa.block_sparse_attention_tiled(q, k, v, grid, tiles, choice, idx, cnt, return_lse=True)
    got = vsa.block_sparse_attention_tiled_backward(g, q, k, v, o, lse, grid, tiles, choice, idx, cnt)
    qp, kp, vp, gp = (vsa.permute(x, grid, tiles, choice) for x in (q, k, v, g))
    op, lp = vsa.block_sparse_attention(qp, kp, vp, idx, cnt, 128, return_lse=True)
    want = vsa.block_sparse_attention_backward(gp, qp, kp, vp, op, lp, idx, cnt, 128)
    for x, y in zip(got, want):
        assert torch.equal(x, vsa.unpermute(y, grid, tiles, choice))


def test_tiled_backward_bad_choice_leaves_the_head():
    grid, tiles, D = (2, 8, 16), [(1, 8, 16)], 64
    q, k, v, g = inputs(1, 2, 256, D, seed=4)
    idx, cnt = random_lists(1, 2, 2, 2, seed=4)
    ok = torch.zeros(2, dtype=torch.int32, device=DEV)
    o, lse = vsa.block_sparse_attention_tiled(q, k, v, grid, tiles, ok, idx, cnt, return_lse=True)
    want = vsa.block_sparse_attention_tiled_backward(g, q, k, v, o, lse, grid, tiles, ok, idx, cnt)
    bad = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    got = vsa.block_sparse_attention_tiled_backward(g, q, k, v, o, lse, grid, tiles, bad, idx, cnt)
    for x, y in zip(got, want):
        assert torch.equal(x[0, 0], y[0, 0])
    with pytest.raises(RuntimeError):
        vsa.device_status()


# --------------------------------------------------------------------------
# windows, with and without a bias
# --------------------------------------------------------------------------

def bucket_of(d, buckets, far):
    """f(d) by whole numbers: bucket e + t starts where d^(n-e) e^t >= e^(n-e) far^t."""
    n = buckets // 2
    e = n // 2
    if d < e:
        return d
    t = 0
    while t < n - 1 - e and d ** (n - e) * e ** (t + 1) >= e ** (n - e) * far ** (t + 1):
        t += 1
    return e + t


@pytest.mark.parametrize("buckets,far", [(32, 128), (4, 2), (6, 100), (16, 5), (64, 2048), (128, 33), (256, 4096), (256, 65)])
def test_relative_position_buckets(buckets, far):
    got = vsa.relative_position_buckets(buckets, far).tolist()
    f = [bucket_of(d, buckets, far) for d in range(far + 1)]
    assert got == [f[-r] for r in range(-far, 1)] + [buckets // 2 + f[r] for r in range(1, far + 1)]


def window_mask(S, window, sink):
    i = torch.arange(S, device=DEV)
    if window >= S:
        return torch.ones(S, S, dtype=torch.bool, device=DEV)
    return (i[None, :] < sink) | ((i[:, None] - i[None, :]).abs() <= window // 2)


@pytest.mark.parametrize("S,D,window,sink,buckets,far,table,scale", [
    (1, 64, 1, 0, 8, 16, torch.float32, None),           # one token
    (2, 128, 1, 1, 4, 2, torch.bfloat16, None),          # a row sees itself and the sink
    (129, 64, 16, 3, 32, 128, torch.bfloat16, None),     # one row in the last tile
    (517, 64, 100, 5, 32, 128, torch.float32, None),
    (640, 128, 256, 0, 16, 20, torch.bfloat16, 0.15),
    (700, 128, 64, 200, 64, 600, torch.float32, None),   # sinks far outside the window
    (900, 64, 5000, 0, 32, 300, torch.bfloat16, None),   # dense
    (1000, 128, 600, 130, 256, 4096, torch.float32, None),
])
def test_window_with_bias(S, D, window, sink, buckets, far, table, scale):
    B, H = 2, 2
    q, k, v, g = inputs(B, H, S, D, seed=S + D)
    gen = torch.Generator(device=DEV).manual_seed(S)
    bias = torch.randn(buckets, H, generator=gen, device=DEV).to(table)
    kw = dict(scale=scale, bias=bias, max_distance=far)
    o, lse = vsa.window_attention(q, k, v, window, sink, return_lse=True, **kw)
    assert torch.equal(o, vsa.window_attention(q, k, v, window, sink, **kw))
    *full, dbias = vsa.window_attention_backward(g, q, k, v, o, lse, window, sink, grad_dtype=torch.float32, **kw)
    again = vsa.window_attention_backward(g, q, k, v, o, lse, window, sink, **kw)
    assert torch.equal(again[3], dbias) and dbias.dtype == table
    for x, y in zip(full, again):
        assert torch.equal(x.to(torch.bfloat16), y)
    f = [bucket_of(d, buckets, far) for d in range(min(S, far) + 1)]
    i = torch.arange(S, device=DEV)
    r = i[None, :] - i[:, None]
    bucket = torch.tensor(f, device=DEV)[r.abs().clamp(max=far)] + (r > 0) * (buckets // 2)
    see = window_mask(S, window, sink)
    want = torch.zeros(buckets, H, dtype=torch.float64, device=DEV)
    err = torch.zeros_like(want)
    for b in range(B):
        for h in range(H):
            ref = reference(q[b, h], k[b, h], v[b, h], g[b, h], see, scale, bias[:, h].double()[bucket])
            assert (lse[b, h].double() - ref["lse"]).abs().max() <= W
            assert ((o[b, h].double() - ref["o"]).abs() <= ref["e_o"] + 1e-6).all()
            check([x[b, h] for x in full], ref, what=f"head {b},{h}")
            want[:, h].index_add_(0, bucket.view(-1), ref["dX"].view(-1))
            err[:, h].index_add_(0, bucket.view(-1), ref["e_dX"].view(-1))
    if table == torch.bfloat16:
        err += U * (want.abs() + err)
    assert ((dbias.double() - want).abs() <= err + 1e-6).all()


@pytest.mark.parametrize("S,D,window,sink", [(1, 128, 1, 0), (130, 64, 7, 0), (391, 128, 120, 140), (512, 64, 512, 0)])
def test_window_backward_without_bias(S, D, window, sink):
    q, k, v, g = inputs(1, 2, S, D, seed=S)
    o, lse = vsa.window_attention(q, k, v, window, sink, return_lse=True)
    assert torch.equal(o, vsa.window_attention(q, k, v, window, sink))
    got = vsa.window_attention_backward(g, q, k, v, o, lse, window, sink, grad_dtype=torch.float32)
    assert len(got) == 3
    for h in range(2):
        check([x[0, h] for x in got], reference(q[0, h], k[0, h], v[0, h], g[0, h], window_mask(S, window, sink)))


def test_zero_bias_changes_nothing_but_rounding():
    q, k, v, g = inputs(1, 2, 300, 64, seed=2)
    bias = torch.zeros(32, 2, device=DEV)
    plain, lse = vsa.window_attention(q, k, v, 64, 3, out_dtype=torch.float32, return_lse=True)
    with_bias, lse2 = vsa.window_attention(q, k, v, 64, 3, out_dtype=torch.float32, bias=bias, return_lse=True)
    # the same sums with the scale applied one rounding earlier (2^-24 of the logit, some of it across a step of P)
    assert (plain - with_bias).abs().max() <= 2 * U * v.abs().max() and (lse - lse2).abs().max() <= 1e-5


# --------------------------------------------------------------------------
# autograd, differences, graphs, streams
# --------------------------------------------------------------------------

def test_gradients_against_differences():
    """<grad, d> against the central difference of the 64-bit loss along random directions d."""
    S, D, window, sink, buckets, far = 200, 64, 40, 3, 16, 32
    q, k, v, g = inputs(1, 1, S, D, seed=6)
    bias = torch.randn(buckets, 1, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    leaves = [x.clone().requires_grad_() for x in (q, k, v)] + [bias.clone().requires_grad_()]
    o = vsa.window_attention(*leaves[:3], window, sink, bias=leaves[3], max_distance=far)
    grads = torch.autograd.grad(o, leaves, g)
    f = [bucket_of(d, buckets, far) for d in range(far + 1)]
    i = torch.arange(S, device=DEV)
    r = i[None, :] - i[:, None]
    bucket = torch.tensor(f, device=DEV)[r.abs().clamp(max=far)] + (r > 0) * (buckets // 2)
    see = window_mask(S, window, sink)

    def loss(q, k, v, b):
        x = (q @ k.T / math.sqrt(D) + b[:, 0][bucket]).masked_fill(~see, -math.inf)
        return (torch.softmax(x, 1) @ v * g[0, 0].double()).sum()

    base = [x[0, 0].double() for x in (q, k, v)] + [bias.double()]
    ref = reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], see, bias=bias[:, 0].double()[bucket])
    errs = [ref["e_dq"], ref["e_dk"], ref["e_dv"],
            torch.zeros(buckets, 1, dtype=torch.float64, device=DEV).index_add_(0, bucket.view(-1), ref["e_dX"].view(-1, 1))]
    for n in range(4):
        d = torch.randn(base[n].shape, dtype=torch.float64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(n))
        e = 1e-5
        up, down = ([x + s * e * d if m == n else x for m, x in enumerate(base)] for s in (1, -1))
        slope = (loss(*up) - loss(*down)) / (2 * e)
        got = grads[n].double().view(d.shape)
        bound = ((errs[n] + U * got.abs()) * d.abs()).sum() + 1e-4
        assert (slope - (got * d).sum()).abs() <= bound
        # the bound is a worst case; a gradient of the wrong sign or size is far outside this one
        assert (slope - (got * d).sum()).abs() <= 0.05 * (got.norm() * d.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_autograd_matches_the_functions(dtype):
    q, k, v, g = inputs(1, 2, 512, 64, seed=7, dtype=dtype)
    idx, cnt = random_lists(1, 2, 4, 3, seed=7)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = vsa.block_sparse_attention(*leaves, idx, cnt, 128)
    with torch.no_grad():
        o2, lse, o_lo = vsa.block_sparse_attention(q, k, v, idx, cnt, 128, return_remainder=True)
        want = vsa.block_sparse_attention_backward(g, q, k, v, o2, lse, idx, cnt, 128, o_lo=o_lo)
        assert (o_lo is None) == (dtype == torch.float32)
    assert torch.equal(o, o2) and o.dtype == dtype
    got = torch.autograd.grad(o, leaves, g)
    for x, y in zip(got, want):
        assert x.dtype == dtype and torch.equal(x, y)
    # an expanded gradient (a sum's) and a backward pass for one leaf alone
    o = vsa.block_sparse_attention(q, leaves[1], v, idx, cnt, 128)
    o.sum().backward()
    ones = vsa.block_sparse_attention_backward(torch.ones_like(o), q, k, v, o2, lse, idx, cnt, 128, o_lo=o_lo)
    assert torch.equal(leaves[1].grad, ones[1]) and q.grad is None


def test_training_step_through_the_compositions():
    """The path as a training step uses it: tiling choice, lists, attention and its gradients."""
    grid, tiles = (4, 16, 16), [(1, 8, 16), (2, 8, 8), (4, 4, 8)]
    q, k, v, g = inputs(1, 2, 1024, 64, seed=11)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    res = {}
    for tiled in (True, False):
        o, mid = vsa.spade_attention(*leaves, grid, tiles, topk=3, tiled=tiled, return_intermediates=True)
        res[tiled] = torch.autograd.grad(o, leaves, g)
    plain = vsa.spade_attention(q, k, v, grid, tiles, topk=3)
    assert torch.equal(o, plain)
    for x, y in zip(res[True], res[False]):
        assert torch.equal(x, y)
    choice, idx, cnt = mid["choice"], mid["idx"], mid["cnt"]
    for h in range(2):
        tok = order_of(grid, tiles[int(choice[h])], grid).to(DEV)
        see = list_mask(idx[0, h], cnt[0, h], 128, 1024)
        at = torch.empty_like(tok)
        at[tok] = torch.arange(1024, device=DEV)
        check([x[0, h] for x in res[True]], reference(q[0, h], k[0, h], v[0, h], g[0, h], see[at][:, at]))


@pytest.mark.parametrize("kind,grid", [("spatial", (2, 8, 16)), ("temporal", (32, 2, 8)), ("temporal", (4, 8, 32)),
                                       ("sliding_tile", (8, 16, 16)), ("sliding_tile_centered", (8, 8, 24))])
def test_structured_attention_backward(kind, grid):
    D, H = 64, 2
    S = math.prod(grid)
    q, k, v, g = inputs(1, H, S, D, seed=S)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = vsa.structured_attention(*leaves, kind, grid)
    assert torch.equal(o, vsa.structured_attention(q, k, v, kind, grid))
    got = torch.autograd.grad(o, leaves, g)
    i = torch.arange(S, device=DEV)
    c = [i // (grid[1] * grid[2]), i // grid[2] % grid[1], i % grid[2]]
    if kind == "spatial":
        see = c[0][:, None] == c[0]
    elif kind == "temporal":
        see = (c[1][:, None] == c[1]) & (c[2][:, None] == c[2])
    else:
        see = torch.ones(S, S, dtype=torch.bool, device=DEV)
        for x, n, t in zip(c, grid, (4, 8, 8)):
            m, a = n // t, x // t
            if kind == "sliding_tile":
                see &= (a[:, None] - a).abs() <= 1
            else:
                w = min(3, m)
                lo = (a - 1).clamp(0, m - w)
                see &= (a[None, :] >= lo[:, None]) & (a[None, :] < lo[:, None] + w)
    for h in range(H):
        check([x[0, h] for x in got], reference(q[0, h], k[0, h], v[0, h], g[0, h], see), what=kind)


def test_permute_gradients():
    grid, tiles = (3, 9, 20), [(1, 8, 16)]
    x = torch.randn(1, 2, 540, 64, device=DEV, requires_grad=True)
    y = vsa.permute(x, grid, tiles)
    g = torch.randn_like(y)
    assert torch.equal(torch.autograd.grad(y, x, g)[0], vsa.unpermute(g, grid, tiles))
    z = torch.randn_like(y).requires_grad_()
    t = vsa.unpermute(z, grid, tiles)
    g = torch.randn_like(t)
    assert torch.equal(torch.autograd.grad(t, z, g)[0], vsa.permute(g, grid, tiles))


def test_calls_in_a_row_repeat_bit_for_bit():
    """Calls right behind one another reuse each other's workspace; a chained kernel that read or wrote too early
    would mix them up."""
    cases = []
    for seed, (nb, longest) in enumerate([(7, 4), (40, 3), (150, 12)]):
        q, k, v, g = inputs(1, 3, nb * 128, 64, seed=seed)
        idx, cnt = random_lists(1, 3, nb, longest, seed=seed)
        table = torch.randn(16, 3, device=DEV)

        def step(q=q, k=k, v=v, g=g, idx=idx, cnt=cnt, table=table):
            o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, 128, return_lse=True)
            a = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, 128)
            o, lse = vsa.window_attention(q, k, v, 300, 20, bias=table, return_lse=True)
            return (*a, *vsa.window_attention_backward(g, q, k, v, o, lse, 300, 20, bias=table),
                    *vsa.transpose_block_lists(idx, cnt))

        cases.append((step, step()))
        torch.cuda.synchronize()
    for _ in range(15):
        for got, want in [(step(), want) for step, want in cases]:
            for x, y in zip(got, want):
                assert torch.equal(x, y)


def test_captured_training_step():
    """A recorded forward and backward pass as one graph, replayed over new values."""
    q, k, v, g = inputs(1, 2, 512, 64, seed=21)
    idx, cnt = random_lists(1, 2, 8, 4, seed=21)
    table = torch.randn(32, 2, device=DEV)
    leaves = [x.requires_grad_() for x in (q, k, v, table)]

    def step():
        o = vsa.block_sparse_attention(*leaves[:3], idx, cnt, 64) + vsa.window_attention(*leaves[:3], 96, bias=leaves[3])
        return (o.detach(), *torch.autograd.grad(o, leaves, g))

    step()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step()
    with torch.no_grad():
        for x, y in zip((q, k, v, g), inputs(1, 2, 512, 64, seed=22)):
            x.copy_(y)
        table.mul_(-1)
    gr.replay()
    got = [x.clone() for x in out]
    for x, y in zip(got, step()):
        assert torch.equal(x, y)


def test_captured_and_on_another_stream():
    q, k, v, g = inputs(1, 2, 700, 64, seed=12)
    bias = torch.randn(32, 2, device=DEV).bfloat16()

    def step():
        o, lse = vsa.window_attention(q, k, v, 128, 9, bias=bias, return_lse=True)
        return (o, *vsa.window_attention_backward(g, q, k, v, o, lse, 128, 9, bias=bias))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graphs = []
    for _ in range(2):  # two graphs, each with its own workspace
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    new = inputs(1, 2, 700, 64, seed=13)
    for x, y in zip((q, k, v, g), new):
        x.copy_(y)
    want = step()
    for gr, _ in graphs:
        gr.replay()
    for _, out in graphs:
        for x, y in zip(out, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("mode", ["lists", "lists64", "one", "tiled", "window", "bias"])
def test_remainder(mode):
    """o + o_lo is the fp32 output to 16 bits, and the gradients are those from the fp32 output to the same."""
    D, H, S = 64, 2, 512
    q, k, v, g = inputs(1, H, S, D, seed=21)
    block = 64 if mode == "lists64" else 128
    idx, cnt = random_lists(1, H, S // block, 1 if mode == "one" else 3, seed=21)
    if mode == "tiled":
        fwd, bwd, args, kw = (vsa.block_sparse_attention_tiled, vsa.block_sparse_attention_tiled_backward,
                              ((4, 8, 16), [(1, 8, 16)], None, idx, cnt), {})
    elif mode in ("window", "bias"):
        fwd, bwd, args = vsa.window_attention, vsa.window_attention_backward, (200, 9)
        kw = dict(bias=torch.randn(32, H, device=DEV)) if mode == "bias" else {}
    else:
        fwd, bwd, args, kw = vsa.block_sparse_attention, vsa.block_sparse_attention_backward, (idx, cnt, block), {}
    o, lse, o_lo = fwd(q, k, v, *args, return_remainder=True, **kw)
    full, lse2 = fwd(q, k, v, *args, out_dtype=torch.float32, return_lse=True, **kw)
    assert torch.equal(o, full.bfloat16()) and torch.equal(lse, lse2)
    # the remainder is at most u |o| and rounded by u of itself
    assert ((o.double() + o_lo.double() - full.double()).abs() <= U * U * full.double().abs()).all()
    low = bwd(g, q, k, v, o, lse, *args, o_lo=o_lo, grad_dtype=torch.float32, **kw)
    want = bwd(g, q, k, v, full, lse, *args, grad_dtype=torch.float32, **kw)
    rough = bwd(g, q, k, v, o, lse, *args, grad_dtype=torch.float32, **kw)
    for x, y, z in zip(low[:3], want, rough):
        # delta differs by u^2 |g||o| where a bf16 o alone would leave u |g||o|; dX and P are rounded alike, so
        # few of their roundings change: u of the gradient's norm is far above what is left
        assert (x - y).norm() <= U / 4 * y.norm()
        assert (z - y).norm() <= 4 * U * y.norm()


def test_bias_without_its_gradient():
    q, k, v, g = inputs(1, 2, 300, 64, seed=14)
    bias = torch.randn(32, 2, device=DEV)
    o, lse = vsa.window_attention(q, k, v, 64, bias=bias, return_lse=True)
    a = vsa.window_attention_backward(g, q, k, v, o, lse, 64, bias=bias)
    b = vsa.window_attention_backward(g, q, k, v, o, lse, 64, bias=bias, bias_grad=False)
    assert b[3] is None
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)
    leaf = q.clone().requires_grad_()
    o, _, o_lo = vsa.window_attention(leaf, k, v, 64, bias=bias, return_remainder=True)
    want = vsa.window_attention_backward(g, q, k, v, o.detach(), lse, 64, bias=bias, bias_grad=False, o_lo=o_lo)
    assert torch.equal(torch.autograd.grad(o, leaf, g)[0], want[0])


@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.float32).min])
def test_bias_that_masks(low):
    """A table entry of the type's lowest value, or -inf, takes its bucket out; a row left without keys is empty."""
    S, D, H, far = 300, 64, 2, 64
    q, k, v, g = inputs(1, H, S, D, seed=31)
    bias = torch.randn(16, H, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    bias[8:, 0] = low    # head 0: no later key
    bias[3, 1] = low     # head 1: one bucket among others (distance 3 backwards)
    bias[0, 1] = bias[1, 1] = 2.0
    f = [bucket_of(d, 16, far) for d in range(far + 1)]
    i = torch.arange(S, device=DEV)
    r = i[None, :] - i[:, None]
    bucket = torch.tensor(f, device=DEV)[r.abs().clamp(max=far)] + (r > 0) * 8
    o, lse, o_lo = vsa.window_attention(q, k, v, 120, 2, bias=bias, max_distance=far, return_remainder=True)
    *grads, dbias = vsa.window_attention_backward(g, q, k, v, o, lse, 120, 2, bias=bias, max_distance=far,
                                                  grad_dtype=torch.float32, o_lo=o_lo)
    vsa.device_status()
    want, err = (torch.zeros(16, H, dtype=torch.float64, device=DEV) for _ in range(2))
    for h in range(H):
        b = bias[:, h].double()
        see = window_mask(S, 120, 2) & (b > -1e30)[bucket]
        ref = reference(q[0, h], k[0, h], v[0, h], g[0, h], see, None, b.clamp(min=-1e30)[bucket])
        check([x[0, h] for x in grads], ref, what=f"head {h}")
        want[:, h].index_add_(0, bucket.view(-1), ref["dX"].view(-1))
        err[:, h].index_add_(0, bucket.view(-1), ref["e_dX"].view(-1))
    assert ((dbias.double() - want).abs() <= err + 1e-6).all()
    assert not dbias[8:, 0].any() and dbias[3, 1] == 0
    # every bucket taken out: every row is empty, nothing is passed on
    bias.fill_(low)
    o, lse = vsa.window_attention(q, k, v, 120, 2, bias=bias, max_distance=far, return_lse=True)
    with pytest.raises(RuntimeError):
        vsa.device_status()
    assert not o.any() and (lse == -math.inf).all()
    out = vsa.window_attention_backward(g, q, k, v, o, lse, 120, 2, bias=bias, max_distance=far)
    assert not any(x.any() for x in out)


def test_non_finite_rows_stay_with_their_neighbours():
    """A NaN in one query's gradient reaches that query, the keys it sees and no other head or block."""
    D, block, nb = 64, 128, 4
    q, k, v, g = inputs(1, 2, nb * block, D, seed=32)
    idx = torch.tensor([[0], [0], [2], [3]], dtype=torch.int32, device=DEV)
    cnt = torch.ones(nb, dtype=torch.int32, device=DEV)
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, return_lse=True)
    clean = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block)
    g[0, 0, 130, 5] = math.nan
    dq, dk, dv = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block)
    assert dq[0, 0, 130].isnan().any()
    for x, y in zip((dq, dk, dv), clean):
        assert torch.equal(x[0, 1], y[0, 1]) and torch.equal(x[0, 0, 2 * block:], y[0, 0, 2 * block:])
    assert torch.equal(dq[0, 0, :block], clean[0][0, 0, :block])
    other = torch.arange(block, 2 * block, device=DEV) != 130
    assert torch.equal(dq[0, 0, block:2 * block][other], clean[0][0, 0, block:2 * block][other])


def test_window_non_finite_rows_stay_alone():
    """A NaN query and a NaN gradient row reach their own dq rows and the keys they see, no other row's dq."""
    S, D = 512, 64
    q, k, v, g = inputs(1, 2, S, D, seed=36)
    bias = torch.randn(16, 2, device=DEV)
    q2, g2 = q.clone(), g.clone()
    q2[0, 0, 200, 3] = math.nan
    g2[0, 0, 210, 3] = math.inf
    out = []
    for qq, gg in ((q, g), (q2, g2)):
        o, lse = vsa.window_attention(qq, k, v, 40, bias=bias, max_distance=30, return_lse=True)
        out.append(vsa.window_attention_backward(gg, qq, k, v, o, lse, 40, bias=bias, max_distance=30))
    others = torch.ones(S, dtype=torch.bool, device=DEV)
    others[200] = others[210] = False
    assert not out[1][0][0, 0, 200].isfinite().all() and not out[1][0][0, 0, 210].isfinite().all()
    # the clean rows' weights of the tiles' means change with the mass of the two rows: rounding only
    assert (out[1][0][0, 0][others] - out[0][0][0, 0][others]).abs().max() <= 2 * U * out[0][0][0, 0].abs().max()
    assert torch.equal(out[1][0][0, 1], out[0][0][0, 1])
    # the tile of queries 128 .. 255 is computed with keys 0 .. 383, where a masked pair is zero times the NaN
    far = torch.arange(S, device=DEV) >= 384
    for x, y in zip(out[1][1:3], out[0][1:3]):
        assert torch.equal(x[0, 0][far], y[0, 0][far]) and torch.equal(x[0, 1], y[0, 1])


@pytest.mark.parametrize("S,window,sink", [(640, 60, 0), (900, 300, 150)])
def test_window_gradients_of_keys_with_a_large_mean(S, window, sink):
    """Keys far from zero and close to one another: dq depends on their spread alone.

    The errors of dX multiply k - c, with c the weighted mean of the tiles' mean keys (fp32 sums of P over a
    quarter of the columns).  With keys m + x, |x| much smaller than |m|, |k_j - c| is at most the largest
    distance of two keys, so the bound of dq takes that in place of |k_j|; the sum of dX that is taken off
    carries fp32 rounding of S terms of size |dX| only, times |c|."""
    D = 64
    q, k, v, g = inputs(1, 1, S, D, seed=S)
    k = (k.float() * 0.25 + 8 * torch.randn(1, 1, 1, D, generator=torch.Generator(device=DEV).manual_seed(1),
                                            device=DEV)).bfloat16()
    q = (q.float() * 0.1).bfloat16()
    o, lse, o_lo = vsa.window_attention(q, k, v, window, sink, return_remainder=True)
    dq = vsa.window_attention_backward(g, q, k, v, o, lse, window, sink, grad_dtype=torch.float32, o_lo=o_lo)[0]
    see = window_mask(S, window, sink)
    ref = reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], see)
    k64 = k[0, 0].double()
    spread = (k64.amax(0) - k64.amin(0))[None, :]
    scale = 1 / math.sqrt(D)
    bound = scale * (ref["e_dX"].sum(1, keepdim=True) * spread
                     + S * 2.0 ** -24 * ref["dX"].abs().sum(1, keepdim=True) * k64.abs().amax(0)[None, :])
    assert ((dq[0, 0].double() - ref["dq"]).abs() <= bound + 1e-5).all()
    # without it the error would be of the size of the mean times the errors of dX
    rough = (scale * ref["e_dX"] @ k64.abs()).norm()
    assert (dq[0, 0].double() - ref["dq"]).norm() <= 0.05 * rough


def check_large_mean(dq, q, k, v, g, see):
    """As for the windows above: dq's errors multiply the keys' spread."""
    S, D = q.shape
    ref = reference(q, k, v, g, see)
    k64 = k.double()
    spread = (k64.amax(0) - k64.amin(0))[None, :]
    scale = 1 / math.sqrt(D)
    bound = scale * (ref["e_dX"].sum(1, keepdim=True) * spread
                     + S * 2.0 ** -24 * ref["dX"].abs().sum(1, keepdim=True) * k64.abs().amax(0)[None, :])
    assert ((dq.double() - ref["dq"]).abs() <= bound + 1e-5).all()
    rough = (scale * ref["e_dX"] @ k64.abs()).norm()
    assert (dq.double() - ref["dq"]).norm() <= 0.05 * rough


def large_mean_inputs(H, S, D):
    q, k, v, g = inputs(1, H, S, D, seed=S + D)
    m = torch.randn(1, H, 1, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    return (q.float() * 0.1).bfloat16(), (k.float() * 0.25 + 8 * m).bfloat16(), v, g


@pytest.mark.parametrize("block,nb,D,longest,group", [(32, 9, 64, 3, 0), (32, 11, 128, 8, 0), (64, 7, 64, 5, 0),
                                                      (64, 6, 128, 1, 0), (128, 5, 128, 3, 0), (128, 4, 64, 2, 64)])
def test_short_lists_gradients_of_keys_with_a_large_mean(block, nb, D, longest, group):
    H = 2
    q, k, v, g = large_mean_inputs(H, block * nb, D)
    idx, cnt = random_lists(1, H, nb, longest, seed=nb)
    if group:  # every row sees a key of its own group: its own block's
        idx = torch.stack([torch.arange(nb), torch.full((nb,), -1)], -1).int().expand(1, H, nb, 2).contiguous().to(DEV)
        cnt = torch.ones(1, H, nb, dtype=torch.int32, device=DEV)
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, group, out_dtype=torch.float32, return_lse=True)
    dq = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block, group, grad_dtype=torch.float32)[0]
    for h in range(H):
        see = list_mask(idx[0, h], cnt[0, h], block, block * nb)
        if group:
            i = torch.arange(block * nb, device=DEV) // group
            see &= i[:, None] == i
        check_large_mean(dq[0, h], q[0, h], k[0, h], v[0, h], g[0, h], see)


@pytest.mark.parametrize("grid,tiles,D", [((3, 9, 17), [(1, 8, 16), (2, 8, 8)], 64), ((5, 6, 12), [(2, 4, 4)], 128),
                                          ((3, 9, 20), [(1, 4, 16), (1, 8, 8)], 128)])
def test_short_tiled_lists_gradients_of_keys_with_a_large_mean(grid, tiles, D):
    """Padding positions hold no key: the mean keys must not count them."""
    H, S, pg = 2, math.prod(grid), vsa.padded_grid(grid, tiles)
    positions, block = math.prod(pg), min(128, math.prod(tiles[0]))
    q, k, v, g = large_mean_inputs(H, S, D)
    choice = (torch.arange(H) % len(tiles)).int().to(DEV)
    idx, cnt = random_lists(1, H, positions // block, 4, seed=S)
    idx[..., 0] = 0  # block 0 holds token 0: no row is without a key
    o, lse = vsa.block_sparse_attention_tiled(q, k, v, grid, tiles, choice, idx, cnt, out_dtype=torch.float32,
                                              return_lse=True)
    dq = vsa.block_sparse_attention_tiled_backward(g, q, k, v, o, lse, grid, tiles, choice, idx, cnt,
                                                   grad_dtype=torch.float32)[0]
    for h in range(H):
        tok = order_of(grid, tiles[int(choice[h])], pg).to(DEV)
        at = torch.empty(S, dtype=torch.long, device=DEV)
        at[tok[tok >= 0]] = torch.arange(positions, device=DEV)[tok >= 0]
        check_large_mean(dq[0, h], q[0, h], k[0, h], v[0, h], g[0, h],
                         list_mask(idx[0, h], cnt[0, h], block, positions)[at][:, at])


@pytest.mark.parametrize("block,nb,longest", [(32, 260, 30), (128, 140, 9)])
def test_backward_over_many_blocks(block, nb, longest):
    """More than 128 blocks: the lists are turned in global memory.  Sampled against the dense formula."""
    D, S = 64, block * nb
    q, k, v, g = inputs(1, 1, S, D, seed=nb)
    idx, cnt = random_lists(1, 1, nb, longest, seed=nb)
    idx[..., 0] = 0  # one block that every query block lists, as a sink is
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, block, return_lse=True)
    got = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, block, grad_dtype=torch.float32)
    see = list_mask(idx[0, 0], cnt[0, 0], block, S)
    check([x[0, 0] for x in got], reference(q[0, 0], k[0, 0], v[0, 0], g[0, 0], see))


def test_two_streams_at_once():
    q, k, v, g = inputs(1, 2, 1024, 64, seed=33)
    idx, cnt = random_lists(1, 2, 8, 5, seed=33)
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, 128, return_lse=True)
    want = vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, 128)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                out.append(vsa.block_sparse_attention_backward(g, q, k, v, o, lse, idx, cnt, 128))
    torch.cuda.synchronize()
    for res in out:
        for x, y in zip(res, want):
            assert torch.equal(x, y)


def test_mixed_input_types():
    """An fp32 q beside bf16 k and v: each gradient in its input's type, from the same roundings."""
    q, k, v, g = inputs(1, 2, 256, 64, seed=34)
    leaves = [q.float().requires_grad_(), k.clone().requires_grad_(), v.clone().requires_grad_()]
    o = vsa.window_attention(*leaves, 64, 2, out_dtype=torch.bfloat16)
    got = torch.autograd.grad(o, leaves, g)
    o2, lse, o_lo = vsa.window_attention(q, k, v, 64, 2, return_remainder=True)
    want = vsa.window_attention_backward(g, q, k, v, o2, lse, 64, 2, o_lo=o_lo, grad_dtype=torch.float32)
    assert torch.equal(o, o2) and [x.dtype for x in got] == [torch.float32, torch.bfloat16, torch.bfloat16]
    for x, y in zip(got, want):
        assert torch.equal(x, y.to(x.dtype))


def test_backward_of_a_backward_is_refused():
    q, k, v, g = inputs(1, 1, 128, 64, seed=35)
    leaf = q.requires_grad_()
    o = vsa.window_attention(leaf, k, v, 64)
    (grad,) = torch.autograd.grad(o, leaf, g, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(grad.sum(), leaf)


def test_refusals():
    q, k, v, g = inputs(1, 2, 256, 64, seed=15)
    idx, cnt = random_lists(1, 2, 2, 2, seed=15)
    o, lse = vsa.block_sparse_attention(q, k, v, idx, cnt, 128, return_lse=True)
    back = vsa.block_sparse_attention_backward
    with pytest.raises(ValueError, match="shape"):
        back(g[:, :, :128], q, k, v, o, lse, idx, cnt, 128)
    with pytest.raises(ValueError, match="contiguous"):
        back(g.transpose(1, 2).contiguous().transpose(1, 2), q, k, v, o, lse, idx, cnt, 128)
    with pytest.raises(ValueError, match="lse"):
        back(g, q, k, v, o, lse.double(), idx, cnt, 128)
    with pytest.raises(ValueError, match="lse"):
        back(g, q, k, v, o, lse[:, :1].contiguous(), idx, cnt, 128)
    with pytest.raises(ValueError, match="idx and cnt"):
        back(g, q, k, v, o, lse, idx[:, :, :1].contiguous(), cnt, 128)
    with pytest.raises(ValueError, match="block"):
        back(g, q, k, v, o, lse, idx, cnt, 96)
    with pytest.raises(ValueError, match="CUDA"):
        back(g, q, k, v, o, lse, idx, cnt.cpu(), 128)
    with pytest.raises(ValueError, match="buckets"):
        vsa.window_attention(q, k, v, 64, bias=torch.zeros(7, 2, device=DEV))
    with pytest.raises(ValueError, match="max_distance"):
        vsa.window_attention(q, k, v, 64, bias=torch.zeros(32, 2, device=DEV), max_distance=8)
    with pytest.raises(ValueError, match="buckets by heads"):
        vsa.window_attention(q, k, v, 64, bias=torch.zeros(2, 32, device=DEV))
    with pytest.raises(ValueError, match="float32"):
        vsa.window_attention(q, k, v, 64, bias=torch.zeros(32, 2, device=DEV).half())
    with pytest.raises(ValueError):
        vsa.relative_position_buckets(32, 0)
    with pytest.raises(ValueError):
        vsa.transpose_block_lists(idx, cnt[..., :1])
