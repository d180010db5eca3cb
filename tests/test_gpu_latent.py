"""Attention over paged latent caches (kvd_attend_latent) and the latent append
against plain 64-bit forms: lengths of zero, one and around every tile and page
border, odd pages, drafted tokens, offsets, garbage in unused slots, refused
sequences and pages, graphs, streams."""
import math

import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


def attend(kvd, c, **kw):
    lse = torch.full(c.ql.shape[:3], math.nan, device=c.device)
    out = torch.full_like(c.ql, math.nan)
    status = kvd.status_tensor()
    kvd.attend_latent(c.ql, c.qr, c.latent, c.rope, c.table, c.seq_lens, c.scale,
                      seq_offset=c.seq_offset, out=out, lse=lse, dev_status=status, **kw)
    return out, lse, int(status.item())


def same(kvd, c, what, drop=(), status=0):
    out, lse, bits = attend(kvd, c)
    assert bits == status, f"{what}: device status {bits}"
    o, z, A, d = c.reference(drop)
    ref.check(what, out, lse, o, z, A, d, max(max(c.lens), 1), c.dtype)


# lens, T, H, R, BS
SHAPES = [
    ([1], 1, 1, 512, 128),
    ([0, 1, 2, 3, 0], 3, 4, 512, 16),
    ([63, 64, 65, 127, 128, 129], 1, 16, 512, 64),
    ([31, 32, 33, 191, 192, 193], 2, 5, 256, 48),
    ([700, 1, 333], 4, 32, 512, 128),
    ([260, 90], 1, 128, 512, 64),
    ([77, 1030], 1, 100, 384, 32),
    ([150, 19], 7, 9, 128, 16),
    ([100, 55, 13], 2, 3, 512, 7),
    ([500, 131], 1, 20, 256, 200),
    ([300], 5, 13, 128, 12),
    ([90, 40], 1, 33, 512, 1),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"T{s[1]}H{s[2]}R{s[3]}BS{s[4]}")
def test_shapes(kvd, shape, dtype):
    lens, T, H, R, BS = shape
    same(kvd, ref.LatentCase(lens, T, H, R, BS, dtype, seed=H + T), "shape")


def test_long_and_many(kvd):
    """One long sequence over the whole grid; many sequences, most of them short."""
    same(kvd, ref.LatentCase([20011], 1, 16, 512, 128, BF, seed=1), "long")
    lens = [(i * 37) % 211 for i in range(400)] + [3001]
    same(kvd, ref.LatentCase(lens, 1, 8, 256, 32, BF, seed=2), "many")
    same(kvd, ref.LatentCase(lens, 2, 4, 128, 32, F32, seed=3), "many f32")


def test_offsets(kvd):
    c = ref.LatentCase([200, 64, 5], 2, 16, 512, 64, BF, seed=4, offsets=[3, 0, 9])
    same(kvd, c, "offset")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_growing_scores(kvd, dtype):
    """The running maximum rises with almost every tile, far beyond 2^8 at once,
    and then falls."""
    c = ref.LatentCase([900, 450], 2, 16, 256, 64, dtype, seed=5)
    for b, (rows, r) in enumerate(c.rows):
        n = rows.shape[0]
        ramp = torch.linspace(0, 12, n, device="cuda").double()
        ramp[2 * n // 3:] = 0.5
        new = (c.ql[b, 0, 0].double()[None] * ramp[:, None] * 0.25 + rows * 0.1).to(dtype)
        rows.copy_(new.double())
        pages = c.table[b, : -(-n // c.BS)].long()
        flat = c.latent[pages].reshape(-1, c.R)
        flat[:n] = new
        c.latent[pages] = flat.view(-1, c.BS, 1, c.R)
    same(kvd, c, "growing")


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.5])
def test_scales(kvd, scale):
    c = ref.LatentCase([130, 71], 1, 16, 256, 32, BF, seed=6)
    c.scale = scale
    same(kvd, c, "scale")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_dropped_pages(kvd, dtype):
    """A page id outside the cache drops that page's tokens; all pages dropped: an
    empty row."""
    c = ref.LatentCase([300, 200, 40], 2, 8, 256, 32, dtype, seed=7)
    NB = c.latent.shape[0]
    c.table[0, 2], c.table[1, 6], c.table[2, 0], c.table[2, 1] = -1, NB, NB + 5, -9
    same(kvd, c, "dropped", drop=[(0, 2), (1, 6), (2, 0), (2, 1)], status=kvd.DEV_BLOCK_RANGE)


def test_refused_sequences(kvd):
    c = ref.LatentCase([100, 200, 70, 90], 1, 4, 128, 32, BF, seed=8)
    cols = c.table.shape[1]
    ends = c.seq_lens.clone()
    c.seq_offset[1] = 32 * (cols - 1)         # sequence 1 runs past the table
    c.seq_offset[3] = 16                      # not a whole page
    out, lse, bits = attend(kvd, c)
    assert bits == kvd.DEV_TABLE_COLS | kvd.DEV_SEQ_OFFSET
    o, z, A, d = c.reference()
    for b in (1, 3):
        o[b], z[b], A[b], d[b] = 0, -math.inf, 0, 0
    ref.check("refused", out, lse, o, z, A, d, 200, BF)
    c.seq_offset.zero_()
    c.seq_lens[2] = ends[3] + 5               # sequence 2 would have a negative length
    out, lse, bits = attend(kvd, c)
    assert bits & kvd.DEV_SEQLENS
    assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())
    c.seq_lens.copy_(ends)
    c.seq_lens[0] = 1                         # does not start at 0
    out, lse, bits = attend(kvd, c)
    assert bits == kvd.DEV_SEQLENS and bool(torch.isneginf(lse[0]).all())


def test_nan_query_stays_in_its_row(kvd):
    c = ref.LatentCase([130, 71], 1, 16, 256, 32, BF, seed=9)
    clean, _, _ = attend(kvd, c)
    c.ql[0, 0, 3, 5] = math.nan
    out, lse, _ = attend(kvd, c)
    assert bool(torch.isnan(out[0, 0, 3]).all()) and bool(torch.isnan(lse[0, 0, 3]))
    keep = torch.ones(2, 1, 16, dtype=torch.bool, device="cuda")
    keep[0, 0, 3] = False
    assert torch.equal(out[keep], clean[keep])


def test_repeatable_and_workspace_content_is_free(kvd):
    c = ref.LatentCase([1500, 900, 20], 2, 16, 512, 64, BF, seed=10)
    need = kvd.attend_latent_workspace_bytes(3, 2, 16, 64, c.table.shape[1], 512, 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    a, la, _ = attend(kvd, c, workspace=ws)
    b, lb, _ = attend(kvd, c, workspace=ws)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_graph_streams_and_new_lengths(kvd):
    """One captured call replayed over other lengths and pages; two streams at
    once with a workspace each."""
    c = ref.LatentCase([400, 31], 1, 16, 256, 32, BF, seed=11, spare=30)
    need = kvd.attend_latent_workspace_bytes(2, 1, 16, 32, c.table.shape[1], 256, 64)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = torch.empty_like(c.ql)
    lse = torch.empty(2, 1, 16, device="cuda")
    args = (c.ql, c.qr, c.latent, c.rope, c.table, c.seq_lens, c.scale)
    kvd.attend_latent(*args, out=out, lse=lse, workspace=ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.attend_latent(*args, out=out, lse=lse, workspace=ws[0])
    for lens in ([400, 31], [0, 31], [77, 1]):
        c.seq_lens.copy_(torch.tensor([0, lens[0], lens[0] + lens[1]], dtype=torch.int32))
        c.lens = lens
        kept, c.rows = c.rows, [(x[:n], y[:n]) for (x, y), n in zip(c.rows, lens)]
        graph.replay()
        torch.cuda.synchronize()
        o, z, A, d = c.reference()
        ref.check("replay", out, lse, o, z, A, d, 400, BF)
        c.rows = kept
    want = out.clone()
    outs = [torch.empty_like(out) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, x in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                kvd.attend_latent(*args, out=x, workspace=w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("BS", [1, 7, 16, 128])
def test_append(kvd, BS, dtype):
    g = torch.Generator().manual_seed(BS)
    new, pos, R, P = [1, 0, 130, 17, 0], [5, 3, 0, 250, 2], 384, 64
    Q, NB, cols = len(new), 400, -(-300 // BS) + 2
    NB = Q * cols + 2
    table = torch.randperm(NB, generator=g)[: Q * cols].view(Q, cols).to(torch.int32)
    off = torch.tensor([0, 0, BS, 0, 0], dtype=torch.int32)
    latent = torch.randn(NB, BS, 1, R, generator=g).to(dtype)
    rope = torch.randn(NB, BS, 1, P, generator=g).to(dtype)
    N = sum(new) + 3                        # three rows behind the last sequence
    cn, rn = torch.randn(N, R, generator=g).to(dtype), torch.randn(N, P, generator=g).to(dtype)
    lens = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    wl, wr = latent.clone(), rope.clone()
    for b in range(Q):
        for i in range(new[b]):
            t = pos[b] + i
            page = int(table[b, int(off[b]) // BS + t // BS])
            wl[page, t % BS, 0], wr[page, t % BS, 0] = cn[lens[b] + i], rn[lens[b] + i]
    dl, dr = latent.cuda(), rope.cuda()
    status = kvd.status_tensor()
    kvd.append_latent(dl, dr, table.cuda(), off.cuda(), cn.cuda(), rn.cuda(), lens.cuda(),
                      torch.tensor(pos, dtype=torch.int32).cuda(), status)
    assert int(status.item()) == 0
    assert torch.equal(dl.cpu(), wl) and torch.equal(dr.cpu(), wr)


def test_append_refusals_on_the_device(kvd):
    """Each bad sequence keeps its pages; the others are written."""
    BS, R, P, NB, cols = 4, 64, 8, 12, 3
    table = torch.arange(12, dtype=torch.int32).view(4, 3)
    table[3, 0] = NB
    latent, rope = torch.zeros(NB, BS, 1, R, device="cuda"), torch.zeros(NB, BS, 1, P, device="cuda")
    cn, rn = torch.ones(8, R, device="cuda"), torch.ones(8, P, device="cuda")
    lens = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32).cuda()
    pos = torch.tensor([-1, 11, 0, 0], dtype=torch.int32).cuda()   # 1: the second row is past cols
    off = torch.tensor([0, 0, 2, 0], dtype=torch.int32).cuda()
    status = kvd.status_tensor()
    kvd.append_latent(latent, rope, table.cuda(), off, cn, rn, lens, pos, status)
    assert int(status.item()) == (kvd.DEV_POS_RANGE | kvd.DEV_TABLE_COLS | kvd.DEV_SEQ_OFFSET
                                  | kvd.DEV_BLOCK_RANGE)
    want = torch.zeros_like(latent)
    want[5, 3] = 1
    assert torch.equal(latent, want) and int(rope.sum().item()) == P
    status.zero_()
    lens = torch.tensor([0, 2, 1, 6, 9], dtype=torch.int32).cuda()  # decreasing; past N
    kvd.append_latent(latent, rope, table.cuda(), None, cn, rn, lens, pos.clamp(min=0), status)
    assert int(status.item()) & kvd.DEV_SEQLENS
