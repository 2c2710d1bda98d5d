"""Argument checks of the Python binding, on the CPU: tensors stand in for CUDA tensors and a
launch that is reached is recorded in place of being made."""

import math

import pytest
import torch

import block_sparse_self_b200 as vsa


class Launched(Exception):
    pass


class Recorder:
    """libvsa with every call that would launch something replaced by the exception above."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name == "vsa_padded_grid" or name.endswith("workspace_size") or name == "vsa_last_error":
            return getattr(self.real, name)

        def launch(*args):
            raise Launched(name)
        return launch


@pytest.fixture
def host(monkeypatch):
    real = vsa.lib()
    monkeypatch.setattr(vsa, "_cuda", lambda t, name: t)
    monkeypatch.setattr(vsa, "lib", lambda: Recorder(real))
    monkeypatch.setattr(vsa, "_stream", lambda device=None: 0)
    monkeypatch.setattr(vsa, "_on", lambda t: vsa._NO_GUARD)


def qkv(B, H, S, D=64, **kw):
    return [torch.zeros(B, H, S, D, dtype=torch.bfloat16, **kw) for _ in range(3)]


def lists(*lead, cap=2):
    return torch.zeros(*lead, cap, dtype=torch.int32), torch.ones(*lead, dtype=torch.int32)


B, H, NB = 2, 3, 4
GRID, TILES = (4, 8, 16), [(1, 8, 16)]
BAD = {
    "too few blocks": lists(B, H, NB - 1),
    "too many blocks": lists(B, H, NB + 1),
    "too few heads": lists(B, H - 1, NB),
    "batch and heads exchanged": lists(H, B, NB),
    "a list per head without the batch": lists(H, NB),
    "a short shared list": lists(NB - 1),
    "a short cnt": (lists(B, H, NB)[0], torch.ones(B, H, NB - 1, dtype=torch.int32)),
    "a cnt of one head": (lists(B, H, NB)[0], torch.ones(NB, dtype=torch.int32)),
    "cnt in another order": (lists(B, H, NB)[0], torch.ones(B, NB, H, dtype=torch.int32)),
    "one row": (torch.zeros(NB, dtype=torch.int32), torch.ones(NB, dtype=torch.int32)),
}
GOOD = {"per head": lists(B, H, NB), "shared": lists(NB), "shared, 3-D": lists(1, NB),
        "flat counts": (lists(B, H, NB)[0], torch.ones(B * H * NB, dtype=torch.int32))}


def calls(q, k, v):
    lse, x = torch.zeros(B, H, q.shape[2]), q
    leaf = q.clone().requires_grad_()
    yield "plain", lambda i, c: vsa.block_sparse_attention(q, k, v, i, c, 128)
    yield "lse", lambda i, c: vsa.block_sparse_attention(q, k, v, i, c, 128, return_lse=True)
    yield "autograd", lambda i, c: vsa.block_sparse_attention(leaf, k, v, i, c, 128)
    yield "backward", lambda i, c: vsa.block_sparse_attention_backward(x, q, k, v, x, lse, i, c, 128)
    yield "tiled", lambda i, c: vsa.block_sparse_attention_tiled(q, k, v, GRID, TILES, None, i, c)
    yield "tiled lse", lambda i, c: vsa.block_sparse_attention_tiled(q, k, v, GRID, TILES, None, i, c, return_lse=True)
    yield "tiled autograd", lambda i, c: vsa.block_sparse_attention_tiled(leaf, k, v, GRID, TILES, None, i, c)
    yield "tiled backward", lambda i, c: vsa.block_sparse_attention_tiled_backward(x, q, k, v, x, lse, GRID, TILES, None,
                                                                                   i, c)
    yield "compensated", lambda i, c: vsa.centroid_compensated_attention(q, k, v, i, c)
    yield "compensated tiled", lambda i, c: vsa.centroid_compensated_attention_tiled(q, k, v, GRID, TILES, None, i, c)


@pytest.mark.parametrize("call", [name for name, _ in calls(*qkv(B, H, 512))])
def test_lists_of_another_shape_are_refused(host, call):
    """Every list call indexes nb rows per head of idx and cnt: fewer would be read past their end."""
    q, k, v = qkv(B, H, math.prod(GRID))
    run = dict(calls(q, k, v))[call]
    for what, (idx, cnt) in BAD.items():
        with pytest.raises(ValueError, match="idx and cnt"):
            run(idx, cnt)
            pytest.fail(what)
    for what, (idx, cnt) in GOOD.items():
        with pytest.raises(Launched):
            run(idx, cnt)


def test_blocks_of_the_padded_grid_are_counted(host):
    """A grid that the tiles do not divide has the lists of its padded grid."""
    grid = (3, 7, 20)                       # padded to (3, 8, 32): 6 blocks
    q, k, v = qkv(1, 1, math.prod(grid))
    for lse in (False, True):
        with pytest.raises(ValueError, match="nb = 6"):
            vsa.block_sparse_attention_tiled(q, k, v, grid, TILES, None, *lists(1, 1, 4), return_lse=lse)
        with pytest.raises(Launched):
            vsa.block_sparse_attention_tiled(q, k, v, grid, TILES, None, *lists(1, 1, 6), return_lse=lse)


@pytest.mark.parametrize("block", [0, -128, 48, 96, 256])
def test_block_sizes_that_are_refused(host, block):
    q, k, v = qkv(1, 1, 768)
    for lse in (False, True):
        with pytest.raises(ValueError, match="block"):
            vsa.block_sparse_attention(q, k, v, *lists(1, 1, 6), block, return_lse=lse)


@pytest.mark.parametrize("compensate", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tiled_spade_attention_gives_bfloat16_unless_told(host, monkeypatch, dtype, compensate):
    """Inputs in fp32 are rounded to bf16 on the way in; the output type is bf16 unless out_dtype says otherwise."""
    asked = []

    def attention(q, k, v, grid, tiles, choice, idx, cnt, scale, out_dtype):
        asked.append(vsa._out_dtype(out_dtype, q))
        return q

    for name in ("block_summaries_tiled", "block_scores", "_select_blocks"):
        monkeypatch.setattr(vsa, name, lambda *a: (None, None))
    monkeypatch.setattr(vsa, "block_sparse_attention_tiled", attention)
    monkeypatch.setattr(vsa, "centroid_compensated_attention_tiled", attention)
    q, k, v = (x.to(dtype) for x in qkv(1, 1, math.prod(GRID)))
    vsa.spade_attention(q, k, v, GRID, TILES, topk=1, compensate=compensate)
    vsa.spade_attention(q, k, v, GRID, TILES, topk=1, compensate=compensate, out_dtype=torch.float32)
    assert asked == [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("tiled", [False, True])
def test_going_back_through_compensated_attention_is_an_error(host, monkeypatch, tiled):
    """Beside other terms of a loss a result without a graph would train with a gradient missing."""
    class Fills(Recorder):
        def __getattr__(self, name):
            if name in ("vsa_centroid_compensated_attention", "vsa_centroid_compensated_attention_tiled"):
                return lambda *args: vsa.OK
            return super().__getattr__(name)

    real = vsa.lib().real
    monkeypatch.setattr(vsa, "lib", lambda: Fills(real))
    q, k, v = qkv(B, H, math.prod(GRID))
    leaf = q.clone().requires_grad_()
    tail = (GRID, TILES, None, *lists(B, H, NB)) if tiled else lists(B, H, NB)
    call = vsa.centroid_compensated_attention_tiled if tiled else vsa.centroid_compensated_attention
    o = call(leaf, k, v, *tail)
    with pytest.raises(NotImplementedError, match="compensated"):
        (o.float().sum() + leaf.float().sum()).backward()
    # without recording, and for inputs that need no gradient, nothing changes
    with torch.no_grad():
        assert not call(leaf, k, v, *tail).requires_grad
    assert not call(q, k, v, *tail).requires_grad
    with pytest.raises(ValueError, match="idx and cnt"):
        call(leaf, k, v, *(GRID, TILES, None) if tiled else (), *lists(B, H, NB - 1))


@pytest.mark.parametrize("call", ["lists", "tiled", "window"])
@pytest.mark.parametrize("what", [1, 2])
def test_going_back_through_lse_or_the_remainder_is_an_error(host, monkeypatch, call, what):
    """A term of the loss that uses them would otherwise train with its gradient missing."""
    class Fills(Recorder):
        def __getattr__(self, name):
            if name in ("vsa_block_sparse_attention_lse", "vsa_block_sparse_attention_tiled_lse",
                        "vsa_window_attention_lse"):
                return lambda *args: vsa.OK
            return super().__getattr__(name)

    real = vsa.lib().real
    monkeypatch.setattr(vsa, "lib", lambda: Fills(real))
    q, k, v = qkv(B, H, math.prod(GRID))
    leaf = q.clone().requires_grad_()
    kw = dict(return_lse=True, return_remainder=True)
    if call == "lists":
        out = vsa.block_sparse_attention(leaf, k, v, *lists(B, H, NB), 128, **kw)
    elif call == "tiled":
        out = vsa.block_sparse_attention_tiled(leaf, k, v, GRID, TILES, None, *lists(B, H, NB), **kw)
    else:
        out = vsa.window_attention(leaf, k, v, 64, **kw)
    with pytest.raises(NotImplementedError, match="lse"):
        (out[0].float().sum() + out[what].float().sum() + leaf.float().sum()).backward()


class Devices:
    """_on() that remembers whose device is current."""

    def __init__(self):
        self.current = []

    def __call__(self, t):
        self.tensor = t
        return self

    def __enter__(self):
        self.current.append(self.tensor)

    def __exit__(self, *a):
        self.current.pop()


@pytest.mark.parametrize("call", ["lists", "tiled", "window", "permute", "unpermute"])
def test_training_calls_launch_with_their_tensors_device_current(host, monkeypatch, call):
    """A stream belongs to a device: with another one current a launch on it fails.  Every launch of a recorded call
    over fp32 inputs, the casts to bf16 among them, is made with the tensors' device current."""
    on, launched = Devices(), []

    class Runs(Recorder):
        def __getattr__(self, name):
            if name == "vsa_padded_grid" or name.endswith("workspace_size"):
                return getattr(self.real, name)

            def launch(*args):
                assert on.current, name
                launched.append(name)
                return vsa.OK
            return launch

    real = vsa.lib().real
    monkeypatch.setattr(vsa, "lib", lambda: Runs(real))
    monkeypatch.setattr(vsa, "_on", on)
    q, k, v = (x.float().requires_grad_() for x in qkv(B, H, math.prod(GRID)))
    if call == "lists":
        o = vsa.block_sparse_attention(q, k, v, *lists(B, H, NB), 128)
    elif call == "tiled":
        o = vsa.block_sparse_attention_tiled(q, k, v, GRID, TILES, None, *lists(B, H, NB))
    elif call == "window":
        o = vsa.window_attention(q, k, v, 64, bias=torch.zeros(8, H, requires_grad=True), max_distance=16)
    else:
        o = getattr(vsa, call)(q, GRID, TILES)
    forward = len(launched)
    o.sum().backward()
    assert forward >= 1 and len(launched) > forward


def test_tokens_of_the_padded_grid():
    for grid, tiles in (((16, 45, 80), [(1, 8, 16), (2, 8, 8), (4, 4, 8)]), ((3, 7, 20), [(1, 8, 16)]),
                        ((1, 1, 1), [(2, 4, 4), (1, 4, 8)]), ((4, 8, 16), [(1, 8, 16)])):
        assert vsa._padded_tokens(grid, tiles) == math.prod(vsa.padded_grid(grid, tiles))
    for tiles in ([], [(1, 0, 16)], [(0, 0, 0)]):
        with pytest.raises(ValueError):
            vsa._padded_tokens((4, 8, 16), tiles)
        with pytest.raises(ValueError):
            vsa._check_tiled_lists(*lists(1, 1, 4), 1, 1, (4, 8, 16), tiles)
