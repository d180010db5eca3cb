"""kvd_attend_latent above 64 query rows a sequence, where several CTAs take one
tile: row counts around every border, pages of all kinds, growing scores, dropped
pages, empty sequences, splits, graphs."""
import math

import pytest
import torch

import latent_ref as ref
from test_gpu_latent import attend, kvd, same  # noqa: F401

pytestmark = pytest.mark.gpu

BF = torch.bfloat16

# lens, T, H, R, BS
SHAPES = [
    ([1], 1, 65, 512, 64),
    ([0, 1, 64, 65, 0], 1, 128, 512, 128),
    ([127, 128, 129, 193], 2, 40, 256, 16),
    ([300, 2], 3, 27, 512, 8),
    ([500, 77, 1], 1, 96, 256, 24),
    ([90, 333], 1, 113, 512, 40),
    ([260, 90], 1, 129, 512, 32),
    ([100, 640], 2, 128, 512, 48),
    ([61, 200], 5, 77, 256, 200),
    ([80, 130], 1, 70, 512, 4),
    ([80, 130], 1, 128, 256, 66),
    ([80, 130], 1, 128, 128, 64),
    ([33], 200, 4, 512, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"T{s[1]}H{s[2]}R{s[3]}BS{s[4]}")
def test_shapes(kvd, shape):  # noqa: F811
    lens, T, H, R, BS = shape
    same(kvd, ref.LatentCase(lens, T, H, R, BS, BF, seed=H + T), "shape")


def test_long_and_many(kvd):  # noqa: F811
    """One long sequence over the whole grid; many sequences, most of them short."""
    same(kvd, ref.LatentCase([20011], 1, 128, 512, 64, BF, seed=1), "long")
    lens = [(i * 37) % 211 for i in range(300)] + [3001]
    same(kvd, ref.LatentCase(lens, 2, 36, 256, 32, BF, seed=2), "many")


@pytest.mark.parametrize("at", [0, 20, 50, 127])
def test_growing_scores(kvd, at):  # noqa: F811
    """One row's running maximum rises with almost every tile, far beyond 2^8 at
    once, and then falls; the others are ordinary."""
    c = ref.LatentCase([900, 450], 1, 128, 256, 64, BF, seed=5)
    for b, (rows, r) in enumerate(c.rows):
        n = rows.shape[0]
        ramp = torch.linspace(0, 12, n, device="cuda").double()
        ramp[2 * n // 3:] = 0.5
        new = (c.ql[b, 0, at].double()[None] * ramp[:, None] * 0.25 + rows * 0.1).to(BF)
        rows.copy_(new.double())
        pages = c.table[b, : -(-n // c.BS)].long()
        flat = c.latent[pages].reshape(-1, c.R)
        flat[:n] = new
        c.latent[pages] = flat.view(-1, c.BS, 1, c.R)
    same(kvd, c, "growing")


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.5])
def test_scales(kvd, scale):  # noqa: F811
    c = ref.LatentCase([130, 71], 2, 48, 512, 32, BF, seed=6)
    c.scale = scale
    same(kvd, c, "scale")


def test_dropped_pages_and_offsets(kvd):  # noqa: F811
    c = ref.LatentCase([300, 200, 40], 2, 64, 512, 32, BF, seed=7)
    NB = c.latent.shape[0]
    c.table[0, 2], c.table[1, 6], c.table[2, 0], c.table[2, 1] = -1, NB, NB + 5, -9
    same(kvd, c, "dropped", drop=[(0, 2), (1, 6), (2, 0), (2, 1)], status=kvd.DEV_BLOCK_RANGE)
    same(kvd, ref.LatentCase([200, 64, 5], 2, 37, 512, 64, BF, seed=4, offsets=[3, 0, 9]), "offset")


def test_nan_query_stays_in_its_row(kvd):  # noqa: F811
    c = ref.LatentCase([130, 71], 1, 100, 256, 32, BF, seed=9)
    clean, _, _ = attend(kvd, c)
    for row in (3, 20, 99):
        c.ql[0, 0, row, 5] = math.nan
    out, lse, _ = attend(kvd, c)
    keep = torch.ones(2, 1, 100, dtype=torch.bool, device="cuda")
    keep[0, 0, [3, 20, 99]] = False
    assert bool(torch.isnan(out[~keep]).all()) and bool(torch.isnan(lse[~keep]).all())
    assert torch.equal(out[keep], clean[keep])


def test_repeatable_in_a_graph(kvd):  # noqa: F811
    c = ref.LatentCase([1500, 900, 20, 0, 64], 1, 128, 512, 64, BF, seed=10)
    need = kvd.attend_latent_workspace_bytes(5, 1, 128, 64, c.table.shape[1], 512, 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    want, lse, _ = attend(kvd, c, workspace=ws)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            kvd.attend_latent(c.ql, c.qr, c.latent, c.rope, c.table, c.seq_lens, c.scale,
                              seq_offset=c.seq_offset, out=out, workspace=ws)
    for _ in range(50):
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
