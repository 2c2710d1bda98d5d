"""The training operators of sparse video attention: what is timed, and their plain forms.

Three operators, each as a training or inference step of a video transformer calls it:

* block-sparse attention with its backward pass (dQ, dK, dV from key-block lists), in
  tile-contiguous order, in T-major order with a tiling per head, and for structured masks;
* sliding-window attention with sinks and a learned relative position bias by buckets,
  alone (inference) and with its backward pass (dQ, dK, dV and the table's gradient);
* transposed block lists: for each key block the query blocks that list it.

Let x be a row of logits over the keys a query sees, x_j = scale q.k_j (+ table[bucket(j - i), h]),
p = softmax(x), o = sum_j p_j v_j.  With g = dL/do:  dv_j = sum_i p_ij g_i,
dx_ij = p_ij (g_i.v_j - g_i.o_i),  dq_i = scale sum_j dx_ij k_j,  dk_j = scale sum_i dx_ij q_i,
dtable[b, h] = sum over the pairs of bucket b of dx_ij.

The bucket of a relative position r = j - i, with n = buckets / 2, e = n // 2 and
f(d) = d below e, else min(n - 1, e + floor((n - e) ln(d / e) / ln(max_distance / e))), is
f(|r|) + (n if r > 0 else 0).
"""

import math

import torch

own = False  # False: plain torch; True: the calls of block_sparse_self_b200


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # lists of one training step's smallest call: 2 heads of 8 blocks, latency only
        dict(name="lists_tiny", op="lists", B=1, H=2, nb=8, k=2),
        # lists of the adaptive recipe at S = 122880: 24 heads of 960 blocks, k = 96
        dict(name="lists_adaptive", op="lists", B=1, H=24, nb=960, k=96),
        # a few odd blocks: the smallest training step, bound by launches
        dict(name="sparse_tiny", op="sparse", mode="explicit", call="functions", B=1, H=3, grid="7x8x16",
             tiles="1x8x16", block=128, D=64, k=2),
        # 64-token blocks of the recipe's own candidates, permuted order, a batch of two
        dict(name="sparse_block64", op="sparse", mode="explicit", call="autograd", B=2, H=5, grid="15x16x32",
             tiles="1x4x16", block=64, D=64, k=12),
        # the fixed tiling at S = 30720 with 40 heads and a 17 % budget: an ordinary layer
        dict(name="sparse_fixed", op="sparse", mode="explicit", call="autograd", B=1, H=40, grid="20x32x48",
             tiles="1x8x16", block=128, D=128, k=40),
        # adaptive tiling at S = 122880, T-major tensors, a tiling per head (a rank's 6 heads): the longest sequence
        dict(name="tiled_adaptive", op="sparse", mode="tiled", call="functions", B=1, H=6, grid="32x48x80",
             tiles="1x8x16,2x8x8,4x4x8", block=128, D=128, k=96),
        # the 16x45x80 grid that no candidate divides, 64-token tiles: padding keys and rows
        dict(name="tiled_padded64", op="sparse", mode="tiled", call="autograd", B=1, H=4, grid="16x45x80",
             tiles="1x4x16,1x8x8", block=64, D=128, k=60),
        # the sliding-tile mask: one list for every head of a batch of two
        dict(name="sliding_tile", op="sparse", mode="sliding", call="autograd", B=2, H=6, grid="20x32x48",
             tiles="4x8x8", block=128, D=128, k=1),
        # an odd short sequence: inference with a bias, latency
        dict(name="window_tiny", op="window", train=False, B=1, H=3, S=517, D=64, window=100, sink=5,
             buckets=32, max_distance=128),
        # the window layer at S = 30720, 24 heads, inference
        dict(name="window_infer", op="window", train=False, B=1, H=24, S=30720, D=128, window=4096, sink=256,
             buckets=32, max_distance=128),
        # an odd batch in training: ragged last tile, few buckets
        dict(name="window_train_odd", op="window", train=True, B=2, H=5, S=1531, D=64, window=257, sink=7,
             buckets=16, max_distance=64),
        # the window layer at S = 30720 in training, buckets that reach across the window
        dict(name="window_train", op="window", train=True, B=1, H=24, S=30720, D=128, window=4096, sink=256,
             buckets=64, max_distance=2048),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["lists", "explicit", "explicit", "tiled", "tiled", "sliding", "infer", "train", "train"])
    if kind == "lists":
        nb = _spread(rng, 3, 960)
        return dict(op="lists", B=rng.randint(1, 2), H=rng.randint(1, 12), nb=nb, k=_spread(rng, 1, max(1, nb // 8)))
    D = rng.choice([64, 128])
    if kind in ("infer", "train"):
        # a training row that sees one key has gradients of zero: nothing to compare
        S = _spread(rng, 1 if kind == "infer" else 40, 30720)
        n = rng.choice([16, 32, 64, 128])
        return dict(op="window", train=kind == "train", B=rng.randint(1, 2), H=rng.randint(1, 8), S=S, D=D,
                    window=_spread(rng, 1 if kind == "infer" else 16, max(16, min(4096, 2 * S))),
                    sink=rng.randint(0, min(S, 256)), buckets=n, max_distance=_spread(rng, n, 4096))
    if kind == "sliding":
        grid = (4 * rng.randint(1, 5), 8 * rng.randint(1, 4), 8 * rng.randint(1, 6))
        return dict(op="sparse", mode="sliding", call="autograd", B=rng.randint(1, 2), H=rng.randint(1, 6),
                    grid="%dx%dx%d" % grid, tiles="4x8x8", block=128, D=D, k=1)
    block = rng.choice([32, 64, 128, 128, 128])
    cand = {32: ["1x4x8", "2x4x4"], 64: ["1x4x16", "1x8x8", "4x4x4"], 128: ["1x8x16", "2x8x8", "4x4x8"]}[block]
    if kind == "explicit":
        t = cand[0]
        tt, th, tw = (int(x) for x in t.split("x"))
        grid = (tt * rng.randint(1, 20), th * rng.randint(1, 4), tw * rng.randint(1, 3))
        nb = grid[0] * grid[1] * grid[2] // block
        return dict(op="sparse", mode="explicit", call=rng.choice(["functions", "autograd"]), B=rng.randint(1, 2),
                    H=rng.randint(1, 8), grid="%dx%dx%d" % grid, tiles=t, block=block, D=D,
                    k=_spread(rng, 1, max(1, nb // 4)))
    cand = rng.sample(cand, rng.randint(1, len(cand)))
    grid = (rng.randint(4, 20), rng.randint(8, 45), rng.randint(16, 80))
    nb = grid[0] * grid[1] * grid[2] // block
    return dict(op="sparse", mode="tiled", call=rng.choice(["functions", "autograd"]), B=1, H=rng.randint(1, 4),
                grid="%dx%dx%d" % grid, tiles=",".join(cand), block=block, D=D, k=_spread(rng, 1, max(1, nb // 8)))


def _dims(text):
    return tuple(int(x) for x in text.split("x"))


def _tiles(case):
    return [_dims(t) for t in case["tiles"].split(",")]


def _padded(grid, tiles):
    return tuple(-(-g // math.lcm(*(t[a] for t in tiles))) * math.lcm(*(t[a] for t in tiles))
                 for a, g in enumerate(grid))


# ---------------------------------------------------------------------------
# Work: inputs read once, outputs written once, two operations per multiply-add.
# A training step has 2 products of the forward pass and 5 of the backward pass
# (the probabilities are recomputed: keeping them would take S x S values).
# ---------------------------------------------------------------------------

def _window_pairs(S, window, sink):
    if window >= S:
        return S * S
    half, total = window // 2, 0
    for i in range(S):
        lo, hi = max(0, i - half), min(S, i + half + 1)
        total += hi - lo + max(0, min(sink, lo)) + max(0, sink - hi)
    return total


def _sliding_pairs(grid, tile):
    n = [g // t for g, t in zip(grid, tile)]
    seen = [sum(min(m - 1, c + 1) - max(0, c - 1) + 1 for c in range(m)) for m in n]
    return seen[0] * seen[1] * seen[2] * (tile[0] * tile[1] * tile[2]) ** 2


def work(case):
    if case["op"] == "lists":
        BH, nb, k = case["B"] * case["H"], case["nb"], case["k"]
        entries = BH * nb * min(nb, k + 2)
        return {"bytes": 2 * 4 * entries + 4 * BH * (2 * nb + 1), "flops": entries}
    B, H, D = case["B"], case["H"], case["D"]
    if case["op"] == "window":
        S, train = case["S"], case["train"]
        pairs, table = B * H * _window_pairs(S, case["window"], case["sink"]), 2 * H * case["buckets"]
        return {"bytes": 2 * (8 if train else 4) * B * H * S * D + (2 if train else 1) * table,
                "flops": 2 * D * (7 if train else 2) * pairs}
    grid = _dims(case["grid"])
    S = grid[0] * grid[1] * grid[2]
    if case["mode"] == "sliding":
        pairs, lists = B * H * _sliding_pairs(grid, _tiles(case)[0]), 0
    else:
        pg = _padded(grid, _tiles(case))
        nb = pg[0] * pg[1] * pg[2] // case["block"]
        kept = min(nb, case["k"])
        # a list names blocks of the padded grid: its real share is the pairs that count
        real = S / (pg[0] * pg[1] * pg[2])
        pairs, lists = int(B * H * nb * kept * case["block"] ** 2 * real * real), 4 * B * H * nb * (kept + 1)
    return {"bytes": 2 * 8 * B * H * S * D + lists, "flops": 2 * D * 7 * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _smooth(BH, grid, D, g, dev):
    """Q and K as smooth fields over (t, h, w), scaled so that scaled scores have a standard deviation near 3."""
    T, Hg, Wg = grid
    S = T * Hg * Wg
    at = torch.arange(S, device=dev)
    x = torch.stack([(at // (Hg * Wg)) / T, (at // Wg % Hg) / Hg, (at % Wg) / Wg], 1).float()
    out = []
    for _ in range(2):
        y = torch.empty(BH, S, D, device=dev)
        for h in range(BH):
            f = torch.randint(-3, 4, (3, 16), generator=g, device=dev).float()
            f[h % 3] *= 2
            ph = 2 * math.pi * (x @ f)
            y[h] = torch.cat([torch.cos(ph), torch.sin(ph)], 1) @ (torch.randn(32, D, generator=g, device=dev) / 4)
        out.append(y.add_(torch.randn(BH, S, D, generator=g, device=dev), alpha=0.5))
    i = torch.randint(0, S, (2, 4096), generator=g, device=dev)
    s = (out[0][:, i[0]] * out[1][:, i[1]]).sum(-1) / math.sqrt(D)
    a = (3.0 / s.std(dim=1).clamp(min=0.1)).sqrt()[:, None, None]
    return out[0] * a, out[1] * a


def _order(grid, pgrid, tile, dev):
    """Position -> token of the tile-contiguous order over the padded grid; -1 at padding."""
    (T, H, W), (P, Q, R), (a, b, c) = grid, pgrid, tile
    t, h, w = (torch.arange(n, device=dev) for n in pgrid)
    tok = (t[:, None, None] * H + h[None, :, None]) * W + w[None, None, :]
    real = (t < T)[:, None, None] & (h < H)[None, :, None] & (w < W)[None, None, :]
    tok = torch.where(real, tok, torch.full_like(tok, -1))
    return tok.view(P // a, a, Q // b, b, R // c, c).permute(0, 2, 4, 1, 3, 5).reshape(-1)


def _score_lists(q, k, block, kk):
    """Top-k key blocks by min/max summaries, with the sink block and the diagonal: ascending, -1 behind the last."""
    BH, P, D = q.shape
    nb = P // block
    qb, kb = q.view(BH, nb, block, D), k.view(BH, nb, block, D)
    qs = qb.amax(2) + qb.amin(2)
    sc = torch.maximum(qs @ kb.amax(2).transpose(1, 2), qs @ kb.amin(2).transpose(1, 2))
    kk = min(kk, nb)
    on = torch.zeros(BH, nb, nb + 1, dtype=torch.bool, device=q.device)
    on.scatter_(2, sc.topk(kk, dim=2).indices, True)
    on[:, :, 0] = True
    eye = torch.arange(nb, device=q.device)
    on[:, eye, eye] = True
    cap = min(nb, kk + 2)
    ids = torch.where(on[:, :, :nb], eye, nb).sort(dim=2).values[:, :, :cap]
    cnt = on.sum(2)
    return torch.where(ids < nb, ids, -1).int().contiguous(), cnt.int().contiguous()


def _sliding_lists(grid, tile, block, dev):
    n = [g // t for g, t in zip(grid, tile)]
    per = tile[0] * tile[1] * tile[2] // block
    nb = n[0] * n[1] * n[2] * per
    i = torch.arange(nb, device=dev) // per
    c = (i // (n[1] * n[2]), i // n[2] % n[1], i % n[2])
    on = torch.ones(nb, nb, dtype=torch.bool, device=dev)
    for x in c:
        on &= (x[:, None] - x[None, :]).abs() <= 1
    cap = int(on.sum(1).max())
    ids = torch.where(on, torch.arange(nb, device=dev), nb).sort(dim=1).values[:, :cap]
    return torch.where(ids < nb, ids, -1).int().contiguous(), on.sum(1).int().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = dict(case)
    B, H = case["B"], case["H"]
    if case["op"] == "lists":
        # the lists of a training step: block scores with a common trend over the key blocks, so
        # that some key blocks are listed by most query blocks and some by few
        nb = case["nb"]
        q = torch.randn(B * H, nb, 16, generator=g, device=dev)
        k = torch.randn(B * H, nb, 16, generator=g, device=dev) + torch.randn(B * H, 1, 16, generator=g, device=dev)
        idx, cnt = _score_lists(q, k, 1, case["k"])
        st.update(idx=idx.view(B, H, nb, -1), cnt=cnt.view(B, H, nb))
        return st
    D = case["D"]
    if case["op"] == "window":
        S, grid = case["S"], (1, 1, case["S"])
        table = torch.randn(case["buckets"], H, generator=g, device=dev) * 0.5
        st["table"] = table.bfloat16().requires_grad_(case["train"])
    else:
        grid = _dims(case["grid"])
        S = grid[0] * grid[1] * grid[2]
    q, k = (x.bfloat16().view(B, H, S, D) for x in _smooth(B * H, grid, D, g, dev))
    v, do = (torch.randn(B, H, S, D, generator=g, device=dev).bfloat16() for _ in range(2))
    if case["op"] == "sparse":
        tiles, block = _tiles(case), case["block"]
        pg = _padded(grid, tiles)
        choice = torch.randint(0, len(tiles), (B * H,), generator=g, device=dev).int()
        if case["mode"] == "sliding":
            st["idx"], st["cnt"] = _sliding_lists(grid, tiles[0], block, dev)
        else:
            orders = torch.stack([_order(grid, pg, t, dev) for t in tiles])[choice.long()]
            at = orders.clamp(min=0)[:, :, None].expand(-1, -1, D)
            pad = (orders < 0)[:, :, None]
            qp, kp = (x.view(B * H, S, D).float().gather(1, at).masked_fill_(pad, 0.0) for x in (q, k))
            idx, cnt = _score_lists(qp, kp, block, case["k"])
            nb = cnt.shape[1]
            st.update(idx=idx.view(B, H, nb, -1), cnt=cnt.view(B, H, nb))
            if case["mode"] == "explicit":  # the tensors are in tile order already
                q, k = qp.bfloat16().view(B, H, S, D), kp.bfloat16().view(B, H, S, D)
        st.update(choice=choice, tile_of=choice.tolist(), grid_=grid, tiles_=tiles, pgrid_=pg)
    train = case["op"] == "sparse" or case["train"]
    st.update(q=q.requires_grad_(train), k=k.requires_grad_(train), v=v.requires_grad_(train), do=do)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_lists(idx, cnt):
    lead, (nb, cap) = idx.shape[:-2], idx.shape[-2:]
    ids = idx.reshape(-1, nb, cap).long()
    n, dev = ids.shape[0], idx.device
    live = torch.arange(cap, device=dev) < cnt.reshape(n, nb, 1)
    on = torch.zeros(n, nb, nb + 1, dtype=torch.int32, device=dev)
    on.scatter_(2, torch.where(live, ids, nb), 1)
    on = on[:, :, :nb].transpose(1, 2).contiguous()  # [list, key block, query block]
    ends = on.sum(2).cumsum(1)
    start = torch.cat([torch.zeros_like(ends[:, :1]), ends], 1)
    to = torch.where(on > 0, start[:, :nb, None] + on.cumsum(2) - 1, nb * cap)
    rows = torch.full((n, nb * cap + 1), -1, dtype=torch.int32, device=dev)
    rows.scatter_(1, to.view(n, -1), torch.arange(nb, dtype=torch.int32, device=dev).repeat(nb).expand(n, -1))
    return start.int().view(*lead, nb + 1), rows[:, :nb * cap].reshape(*lead, nb * cap)


def _plain_head(q, k, v, do, idx, cnt, block, scale, see, bias):
    """One head in 32 bits: q, k, v, do [P, D] in block order; see(i, j) tells which positions see one another, bias(i, j) adds to the logits; do None: the forward pass alone."""
    P, D = q.shape
    nb, cap = idx.shape
    dev = q.device
    at = idx.clamp(min=0).long()
    i = torch.arange(P, device=dev).view(nb, block, 1)
    j = (at[:, :, None] * block + torch.arange(block, device=dev)).view(nb, 1, cap * block)
    live = (torch.arange(cap, device=dev) < cnt[:, None]).repeat_interleave(block, 1)[:, None, :]
    qb, kb, vb = q.view(nb, block, D), k.view(nb, block, D)[at].view(nb, -1, D), v.view(nb, block, D)[at].view(nb, -1, D)
    x = torch.matmul(qb, kb.transpose(1, 2)).mul_(scale)
    if bias is not None:
        x += bias(i, j)
    if see is not None:
        live = live & see(i, j)
    x.masked_fill_(~live, -math.inf)
    top = x.amax(2, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    p /= p.sum(2, keepdim=True).clamp(min=1e-37)
    o = torch.matmul(p, vb)
    if do is None:
        return (o.view(P, D),)
    gb = do.view(nb, block, D)
    dv = torch.zeros_like(v).view(nb, block * D).index_add_(
        0, at.view(-1), torch.matmul(p.transpose(1, 2), gb).view(nb * cap, block * D))
    dx = torch.matmul(gb, vb.transpose(1, 2)).sub_((gb * o).sum(2, keepdim=True)).mul_(p)
    dq = torch.matmul(dx, kb).mul_(scale)
    dk = torch.zeros_like(k).view(nb, block * D).index_add_(
        0, at.view(-1), torch.matmul(dx.transpose(1, 2), qb).mul_(scale).view(nb * cap, block * D))
    return o.view(P, D), dq.view(P, D), dk.view(P, D), dv.view(P, D), dx


def _plain_buckets(n, far, dev):
    """The bucket of each relative position from -far to far."""
    n //= 2
    e = n // 2
    r = torch.arange(-far, far + 1, device=dev)
    d = r.abs().double()
    log = e + torch.floor((n - e) * torch.log(d.clamp(min=e) / e) / math.log(far / e) + 1e-9)
    return torch.where(d < e, d, log.clamp(max=n - 1)).long() + n * (r > 0)


def _plain_sparse(st):
    q, k, v, do = (st[x].detach() for x in ("q", "k", "v", "do"))
    B, H, S, D = q.shape
    outs = [torch.empty(B * H, S, D, dtype=torch.bfloat16, device=q.device) for _ in range(4)]
    for h in range(B * H):
        at = None if st["mode"] == "explicit" else _order(st["grid_"], st["pgrid_"], st["tiles_"][
            st["tile_of"][h] if st["mode"] == "tiled" else 0], q.device)
        one = [x.view(B * H, S, D)[h].float() for x in (q, k, v, do)]
        if at is not None:
            one = [torch.where((at >= 0)[:, None], x[at.clamp(min=0)], 0.0) for x in one]
        idx, cnt = (x if x.dim() < 3 else x.flatten(0, 1)[h] for x in (st["idx"], st["cnt"])) if (
            st["mode"] != "sliding") else (st["idx"], st["cnt"])
        res = _plain_head(*one, idx, cnt, st["block"], 1 / math.sqrt(D),
                          None if at is None else lambda i, j: (at >= 0)[j], None)[:4]
        for y, r in zip(outs, res):
            if at is None:
                y[h] = r.bfloat16()
            else:  # padding positions go to a row past the last
                y[h] = torch.empty(S + 1, D, dtype=torch.bfloat16, device=q.device).index_copy_(
                    0, torch.where(at >= 0, at, S), r.bfloat16())[:S]
    return [y.view(B, H, S, D) for y in outs]


def _plain_window(st):
    q, k, v, do, table = (st[x].detach() for x in ("q", "k", "v", "do", "table"))
    B, H, S, D = q.shape
    dev, half, sink, far = q.device, st["window"] // 2, st["sink"], st["max_distance"]
    dense = st["window"] >= S
    nb = -(-S // 128)
    # key blocks that the window or the sinks reach, per block of 128 queries
    b = torch.arange(nb, device=dev)
    near = (b[:, None] * 128 - half < (b[None, :] + 1) * 128) & (b[:, None] * 128 + 127 + half >= b[None, :] * 128)
    need = near | (b[None, :] * 128 < sink) | dense
    cap = nb if dense else min(nb, 2 * (-(-half // 128)) + 1 + -(-sink // 128))
    idx = torch.where(need, b, nb).sort(dim=1).values[:, :cap]
    idx, cnt = torch.where(idx < nb, idx, -1), need.sum(1)
    bucket = _plain_buckets(st["buckets"], far, dev)
    outs = [torch.empty(B * H, S, D, dtype=torch.bfloat16, device=dev) for _ in range(4 if st["train"] else 1)]
    dtable = torch.zeros(st["buckets"], H, dtype=torch.float64, device=dev)

    def see(i, j):
        return (j < S) & ((j < sink) | ((i - j).abs() <= half) | dense)

    for h in range(B * H):
        one = [torch.zeros(nb * 128, D, device=dev) for _ in range(4)]
        for x, y in zip(one, (q, k, v, do)):
            x[:S] = y.view(B * H, S, D)[h]
        by = table[:, h % H].float()[bucket]
        if not st["train"]:
            one[3] = None
        res = _plain_head(*one, idx, cnt, 128, 1 / math.sqrt(D), see, lambda i, j: by[(j - i).clamp(-far, far) + far])
        for y, r in zip(outs, res):
            y[h] = r[:S].bfloat16()
        if st["train"]:
            # sums over the diagonals of each pair of blocks (equal j - i): rows reversed, 256 wide,
            # read again 255 wide, put element (r, c) into column 127 - r + c
            dx = res[4].view(nb, 128, cap, 128).transpose(1, 2).flip(2)
            wide = torch.nn.functional.pad(dx, (0, 128)).reshape(nb, cap, 128 * 256)[:, :, :128 * 255]
            diag = wide.view(nb, cap, 128, 255).sum(2, dtype=torch.float64)
            r = (idx[:, :, None] - b[:, None, None]) * 128 + torch.arange(-127, 128, device=dev)
            at = bucket[r.clamp(-far, far) + far]
            dtable[:, h % H].index_add_(0, at.view(-1), diag.view(-1))
    return [y.view(B, H, S, D) for y in outs] + ([dtable.bfloat16()] if st["train"] else [])


def run(st):
    if not own:
        with torch.no_grad():
            if st["op"] == "lists":
                return _plain_lists(st["idx"], st["cnt"])
            if st["op"] == "window":
                return _plain_window(st)
            return _plain_sparse(st)
    import block_sparse_self_b200 as vsa
    if st["op"] == "lists":
        return vsa.transpose_block_lists(st["idx"], st["cnt"])
    q, k, v, do = st["q"], st["k"], st["v"], st["do"]
    if st["op"] == "window":
        kw = dict(bias=st["table"], max_distance=st["max_distance"])
        o = vsa.window_attention(q, k, v, st["window"], st["sink"], **kw)
        return (o, *torch.autograd.grad(o, (q, k, v, st["table"]), do)) if st["train"] else (o,)
    if st["mode"] == "sliding":
        o = vsa.structured_attention(q, k, v, "sliding_tile", st["grid_"], tile=st["tiles_"][0])
        return (o, *torch.autograd.grad(o, (q, k, v), do))
    if st["mode"] == "explicit":
        lists = (st["idx"], st["cnt"], st["block"])
        fwd, bwd = vsa.block_sparse_attention, vsa.block_sparse_attention_backward
    else:
        lists = (st["grid_"], st["tiles_"], st["choice"], st["idx"], st["cnt"])
        fwd, bwd = vsa.block_sparse_attention_tiled, vsa.block_sparse_attention_tiled_backward
    if st["call"] == "autograd":
        o = fwd(q, k, v, *lists)
        return (o, *torch.autograd.grad(o, (q, k, v), do))
    with torch.no_grad():
        o, lse = fwd(q, k, v, *lists, return_lse=True)
        return (o, *bwd(do, q, k, v, o, lse, *lists))


# ---------------------------------------------------------------------------
# The definition in 64 bits, differentiated by autograd
# ---------------------------------------------------------------------------

def _exact_lists(st):
    idx, cnt = st["idx"].cpu().numpy(), st["cnt"].cpu().numpy()
    B, H, nb, cap = idx.shape
    start = torch.zeros(B, H, nb + 1, dtype=torch.int32)
    rows = torch.full((B, H, nb * cap), -1, dtype=torch.int32)
    for b in range(B):
        for h in range(H):
            who = [[] for _ in range(nb)]
            for i in range(nb):
                for j in idx[b, h, i, :cnt[b, h, i]]:
                    who[j].append(i)
            flat = [i for w in who for i in w]
            start[b, h, 1:] = torch.tensor([len(w) for w in who]).cumsum(0).int()
            rows[b, h, :len(flat)] = torch.tensor(flat, dtype=torch.int32)
    return [start, rows]


def _exact_bucket(d, n, e, far):
    """f(d) by whole numbers: d reaches bucket e + t when d^(n-e) e^t >= e^(n-e) far^t."""
    if d < e:
        return d
    t = 0
    while t < n - 1 - e and d ** (n - e) * e ** (t + 1) >= e ** (n - e) * far ** (t + 1):
        t += 1
    return e + t


def _exact_order(grid, pgrid, tile, dev):
    """The same order by sorting the padded grid's cells by the number of their tile."""
    p = torch.arange(pgrid[0] * pgrid[1] * pgrid[2], device=dev)
    t, h, w = p // (pgrid[1] * pgrid[2]), p // pgrid[2] % pgrid[1], p % pgrid[2]
    label = ((t // tile[0]) * (pgrid[1] // tile[1]) + h // tile[1]) * (pgrid[2] // tile[2]) + w // tile[2]
    token = torch.where((t < grid[0]) & (h < grid[1]) & (w < grid[2]), (t * grid[1] + h) * grid[2] + w, -1)
    return token[torch.argsort(label, stable=True)]


def _exact_attention(q, k, v, do, rows, keys_of, mask_of, bias_of, table):
    """softmax attention of row groups in 64 bits and its gradients: rows is a list of index tensors, keys_of(n) the keys that group n may see, mask_of(i, j) what it does see."""
    full = [x.double() for x in (q, k, v)] + ([table.double()] if table is not None else [])
    grads = [torch.zeros_like(x) for x in full]
    o = torch.zeros_like(full[0])
    for n, i in enumerate(rows):
        j = keys_of(n)
        leaves = [x.requires_grad_() for x in (full[0][i], full[1][j], full[2][j])]
        leaves += [x.clone().requires_grad_() for x in full[3:]]
        logits = leaves[0] @ leaves[1].T / math.sqrt(q.shape[1])
        if table is not None:
            logits = logits + bias_of(leaves[3], i, j)
        seen = mask_of(i, j)
        if seen is not None:
            logits = logits.masked_fill(~seen, -math.inf)
        y = torch.softmax(logits, dim=1) @ leaves[2]
        o[i] = y.detach()
        if do is not None:
            part = torch.autograd.grad(y, leaves, do[i].double())
            for total, at, x in zip(grads, (i, j, j), part):
                total.index_add_(0, at, x)
            if table is not None:
                grads[3] += part[3]
    return [o] + (grads if do is not None else [])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "lists":
        return _exact_lists(st)
    q, k, v, do = (st[x].detach().flatten(0, 1) for x in ("q", "k", "v", "do"))
    BH, S, D = q.shape
    dev = q.device
    outs = None
    if case["op"] == "window":
        B, H, half, sink, far = case["B"], case["H"], case["window"] // 2, case["sink"], case["max_distance"]
        dense = case["window"] >= S
        n = case["buckets"] // 2
        f = [_exact_bucket(d, n, n // 2, far) for d in range(far + 1)]
        bucket = torch.tensor([f[-r] for r in range(-far, 1)] + [n + f[r] for r in range(1, far + 1)], device=dev)
        rows = list(torch.arange(S, device=dev).split(1024))
        span = [(max(0, int(i[0]) - half), min(S, int(i[-1]) + half + 1)) for i in rows]
        span = [(0, S) if dense else s for s in span]
        keys = [torch.cat([torch.arange(min(sink, lo)), torch.arange(lo, hi), torch.arange(max(hi, 0), max(hi, sink))]).to(dev)
                for lo, hi in span]
        dtable = torch.zeros(case["buckets"], H, dtype=torch.float64, device=dev)
        for h in range(BH):
            res = _exact_attention(
                q[h], k[h], v[h], do[h] if case["train"] else None, rows, lambda m: keys[m],
                lambda i, j: None if dense else (j[None, :] < sink) | ((i[:, None] - j[None, :]).abs() <= half),
                lambda t, i, j: t[bucket[(j[None, :] - i[:, None]).clamp(-far, far) + far]],
                st["table"].detach()[:, h % H])
            outs = outs or [torch.empty(BH, S, D, dtype=torch.float64, device=dev) for _ in res[:4]]
            for y, r in zip(outs, res):
                y[h] = r
            if case["train"]:
                dtable[:, h % H] += res[4]
        outs = [y.view(case["B"], H, S, D) for y in outs]
        return outs + [dtable] if case["train"] else outs
    block, sliding = case["block"], case["mode"] == "sliding"
    idx, cnt = (x.cpu() for x in (st["idx"], st["cnt"]))
    if not sliding:
        idx, cnt = idx.flatten(0, 1), cnt.flatten(0, 1)
    outs = [torch.empty(BH, S, D, dtype=torch.float64, device=dev) for _ in range(4)]
    for h in range(BH):
        if case["mode"] == "explicit":
            tok = torch.arange(S, device=dev)
        else:
            tok = _exact_order(st["grid_"], st["pgrid_"], st["tiles_"][0 if sliding else int(st["choice"][h])], dev)
        tok = tok.view(-1, block)
        li, lc = (idx, cnt) if sliding else (idx[h], cnt[h])
        rows = [t[t >= 0] for t in tok]
        keep = [n for n, t in enumerate(rows) if t.numel()]

        def keys_of(n):
            t = tok[li[keep[n], :int(lc[keep[n]])].long().to(dev)].reshape(-1)
            return t[t >= 0]

        if len(keep) * BH > 15000:  # a loop over so many groups would take too long
            return None
        res = _exact_attention(q[h], k[h], v[h], do[h], [rows[n] for n in keep], keys_of, lambda i, j: None, None, None)
        for y, r in zip(outs, res):
            y[h] = r
    return [y.view(case["B"], case["H"], S, D) for y in outs]
