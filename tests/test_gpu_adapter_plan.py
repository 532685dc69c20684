"""Adapter calls on plan buffers that hold other words than a plan of the batch:
no access leaves the given buffers, and rows of tiles that a plan of these sizes
cannot hold are left alone."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

GUARD = 4096
TOP = 2 ** 31 - 1


def plan_words(L, T):
    """Offsets (in int32 words) of an adapter plan's parts, and its rows and tiles."""
    up = lambda w: -(-w // 64) * 64  # noqa: E731
    used = min(T, L + 1)
    rows, tiles = -(-(T + 15 * used) // 32) * 32, T // 64 + used
    first = 64
    at_rows = first + up(L + 2)
    return first, at_rows, at_rows + up(rows), rows, tiles


class Guarded:
    """Buffers with a guarded page on either side."""

    def __init__(self):
        self.all = []

    def bytes(self, n, fill=0xA5):
        import torch

        b = torch.full((n + 2 * GUARD,), 0x5C, dtype=torch.uint8, device="cuda")
        b[GUARD:GUARD + n] = fill
        self.all.append((b, n))
        return b[GUARD:GUARD + n]

    def array(self, dtype, *shape):
        n = int(np.prod(shape)) * dtype.itemsize
        return self.bytes(n).view(dtype).view(shape)

    def check(self):
        for b, n in self.all:
            assert bool((b[:GUARD] == 0x5C).all()) and bool((b[GUARD + n:] == 0x5C).all())


# (group, first row, rows) of tiles that no plan of two adapters with `rows` padded rows has
BAD = [lambda rows: (0, TOP - 15, 64), lambda rows: (1, TOP - 63, 64), lambda rows: (0, TOP - 15, 1),
       lambda rows: (3, 0, 16), lambda rows: (-1, 0, 16), lambda rows: (0, 8, 16), lambda rows: (0, -16, 16),
       lambda rows: (0, 0, 0), lambda rows: (0, 0, 65), lambda rows: (0, rows, 1), lambda rows: (0, rows - 16, 17),
       lambda rows: (1, -TOP - 1, TOP)]


@pytest.mark.parametrize("T", [40, 1100])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_tiles_that_no_plan_holds(T, out):
    import torch

    import mixed_precision_moe_topk_amd as M

    L, R, K, N = 2, 20, 136, 72
    d = M.AdapterDims(L, R, K, N, out)
    first, at_rows, at_tiles, rows, tiles = plan_words(L, T)
    words = np.full(M.adapter_plan_query(L, T) // 4, TOP - 15, np.int32)
    words[first:first + L + 2] = [TOP, -TOP, 32, TOP]
    words[at_rows:at_rows + rows:3] = -TOP
    for i in range(tiles):
        words[at_tiles + 4 * i:at_tiles + 4 * i + 3] = BAD[i % len(BAD)](rows)
    assert at_tiles + 4 * tiles <= len(words)

    g = Guarded()
    lo = torch.bfloat16
    ot = lo if out == "bf16" else torch.float32
    for shift in range(0, len(BAD), max(1, tiles)):  # every bad tile, where a batch has few
        for i in range(tiles):
            words[at_tiles + 4 * i:at_tiles + 4 * i + 3] = BAD[(i + shift) % len(BAD)](rows)
        plan = g.bytes(4 * len(words))
        plan.copy_(torch.from_numpy(words.view(np.uint8)))
        ws, saved = g.bytes(M.adapter_workspace_query(d, T)), g.bytes(M.adapter_saved_query(d, T))
        x, a, b = g.array(lo, T, K), g.array(lo, L, R, K), g.array(lo, L, R, N)
        res, dout, dx = g.array(ot, T, N), g.array(ot, T, N), g.array(lo, T, K)
        scale = torch.ones(L, device="cuda")
        before = res.clone(), dx.clone()
        M.adapter_apply(d, x, plan, a, b, scale, dout, res, ws, saved=saved)
        da, db = g.array(torch.float32, L, R, K), g.array(torch.float32, L, R, N)
        M.adapter_backward(d, dout, x, plan, a, b, scale, saved, da, db, ws, dx=dx, dx_base=x)
        torch.cuda.synchronize()
        g.check()
        for got, want in zip((res, dx), before):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
        g.all.clear()
