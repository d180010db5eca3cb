"""kvd_attend_paged_prefix against one softmax in 64 bits over prefix and own tokens;
bounds in latent_ref.py."""
import math

import pytest
import torch

import latent_ref as lref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvd():
    from decode_attention_kv_gb300 import kvd as _kvd
    _kvd.load()
    return _kvd


class Case:
    """Groups of sequences behind prefixes in random pages; every slot that holds no
    token is NaN (keys) or infinite (values)."""

    def __init__(self, groups, pre, own, Hq, Hkv, D, BS, dtype, seed=0, offsets=None, k_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        Q, G = len(own), len(groups)
        self.groups, self.pre, self.own, self.D, self.BS, self.dtype = groups, pre, own, D, BS, dtype
        self.Hq, self.Hkv = Hq, Hkv
        offsets = offsets or [0] * Q
        lists = [(n, 0) for n in pre] + list(zip(own, offsets))
        pages = [-(-n // BS) for n, _ in lists]
        NB = sum(pages) + 3
        order = torch.randperm(NB, generator=g)
        pcols = max([1] + pages[:G]) + 1
        cols = max([1] + [o + p for p, (_, o) in zip(pages[G:], lists[G:])]) + 1
        ptable = torch.full((G, pcols), -3, dtype=torch.int32)
        table = torch.full((Q, cols), -7, dtype=torch.int32)
        kc, vc = torch.full((NB, BS, Hkv, D), math.nan), torch.full((NB, BS, Hkv, D), math.inf)
        self.rows, at = [], 0
        for i, (n, off) in enumerate(lists):
            ids = order[at:at + pages[i]]
            at += pages[i]
            k = (torch.randn(n, Hkv, D, generator=g) * k_scale).to(dtype)
            v = torch.randn(n, Hkv, D, generator=g).to(dtype)
            for j, page in enumerate(ids.tolist()):
                part = slice(j * BS, min(n, (j + 1) * BS))
                kc[page, :part.stop - part.start] = k[part].float()
                vc[page, :part.stop - part.start] = v[part].float()
            if i < G:
                ptable[i, :pages[i]] = ids.to(torch.int32)
            else:
                table[i - G, off:off + pages[i]] = ids.to(torch.int32)
            self.rows.append((k.double().cuda(), v.double().cuda()))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        cum = lambda x: i32([sum(x[:j]) for j in range(len(x) + 1)])  # noqa: E731
        self.ptable, self.table = ptable.cuda(), table.cuda()
        self.kc, self.vc = kc.to(dtype).cuda(), vc.to(dtype).cuda()
        self.q = torch.randn(Q, Hq, D, generator=g).to(dtype).cuda()
        self.plens, self.glens, self.lens = i32(pre), cum(groups), cum(own)
        self.offset = i32([o * BS for o in offsets])
        self.scale = 1.0 / math.sqrt(D)

    def args(self):
        return (self.q, self.kc, self.vc, self.ptable, self.plens, self.glens, self.table,
                self.lens)

    def reference(self, prefix=True, scale=None, drop=()):
        """drop: (list, page) pairs whose tokens do not count (lists: prefixes, then sequences)."""
        Q, Hq, D = self.q.shape
        G, g = len(self.groups), self.Hq // self.Hkv
        of = [i for i, n in enumerate(self.groups) for _ in range(n)]
        out = torch.zeros((Q, Hq, D), dtype=torch.float64, device="cuda")
        A, lse = torch.zeros_like(out), torch.full((Q, Hq), -math.inf, dtype=torch.float64, device="cuda")
        d = torch.zeros_like(lse)
        for b in range(Q):
            lists = ([of[b]] if prefix and b < len(of) else []) + [G + b]
            parts = []
            for i in lists:
                n = self.rows[i][0].shape[0]
                keep = torch.ones(n, dtype=torch.bool, device="cuda")
                for di, page in drop:
                    if di == i:
                        keep &= torch.arange(n, device="cuda") // self.BS != page
                parts.append((self.rows[i][0][keep], self.rows[i][1][keep]))
            k, v = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
            for h in range(self.Hkv):
                hs = slice(h * g, (h + 1) * g)
                seen = torch.ones((g, k.shape[0]), dtype=torch.bool, device="cuda")
                o, z, a, e = lref.attention(self.q[b, hs].double(), k[:, h], v[:, h],
                                            self.scale if scale is None else scale, seen)
                out[b, hs], lse[b, hs], A[b, hs], d[b, hs] = o, z, a, e
        return out, lse, A, d


def same(kvd, c, name, ref=None, bits=0, **kw):
    status, lse = kvd.status_tensor(), torch.full(c.q.shape[:2], 7.0, device="cuda")
    out = kvd.attend_paged_prefix(*c.args(), seq_offset=c.offset, lse=lse, dev_status=status, **kw)
    want = ref or c.reference()
    n = max([0] + c.pre) + max([0] + c.own)
    lref.check(name, out, lse, *want, n, c.dtype)
    assert int(status.item()) == bits
    return out, lse


# groups, prefixes, own lengths, Hq, Hkv, D, BS
SHAPES = [
    ([1], [1], [0], 1, 1, 64, 16),
    ([1], [17], [1], 4, 1, 128, 16),
    ([3], [300], [5, 0, 40], 32, 8, 128, 16),
    ([2, 0, 3], [33, 50, 129], [1, 2, 3, 4, 5], 8, 2, 64, 32),
    ([4, 1], [0, 64], [9, 0, 8, 7, 100], 6, 2, 128, 24),
    ([33], [1000], [i % 7 for i in range(33)], 8, 2, 128, 64),
    ([70], [257], [3 * i % 50 for i in range(70)], 16, 4, 64, 128),
    ([1, 1, 1, 1], [128, 127, 129, 1], [1, 1, 1, 1], 5, 1, 64, 7),
    ([2], [50], [3, 300, 10, 0], 4, 4, 128, 1),         # two sequences behind the groups
    ([3], [700], [20, 10, 30], 48, 1, 128, 48),
    ([2], [2500], [0, 0], 160, 1, 64, 16),              # more heads than a tile has rows
    ([5] * 13, [40 + 10 * i for i in range(13)], [i % 9 for i in range(65)], 8, 4, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"G{len(s[0])}Q{len(s[2])}Hq{s[3]}D{s[5]}BS{s[6]}P{max(s[1])}")
def test_shapes(kvd, shape, dtype):
    same(kvd, Case(*shape, dtype, seed=shape[3]), "shape")


@pytest.mark.parametrize("P", [1, 127, 128, 129, 255, 256, 257, 640, 1025, 5000])
@pytest.mark.parametrize("Q", [1, 20, 40])
def test_lengths(kvd, P, Q):
    """Prefixes that end at and around tile borders, few rows and more than a tile."""
    same(kvd, Case([Q], [P], [i % 3 for i in range(Q)], 8, 2, 128, 16, BF, seed=P), "length")


def test_offsets(kvd):
    same(kvd, Case([2, 2], [40, 50], [20, 30, 0, 70], 8, 2, 64, 16, F32, offsets=[0, 3, 1, 2]), "offset")


def test_large_scores(kvd):
    """Scores that differ by hundreds: the running maximum moves, weights vanish."""
    for dtype in (BF, F32):
        same(kvd, Case([3], [600], [20, 1, 0], 8, 2, 128, 16, dtype, k_scale=20.0), "large")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_scales(kvd, dtype):
    c = Case([2], [200], [9, 30], 8, 2, 64, 16, dtype)
    for scale in (-0.3, 0.0, 1e-35):
        same(kvd, c, f"scale {scale}", ref=c.reference(scale=scale), scale=scale)
    out = kvd.attend_paged_prefix(*c.args(), scale=math.nan)
    assert bool(torch.isnan(out).all())


def test_no_groups_is_the_paged_attention(kvd):
    c = Case([], [], [50, 0, 7], 8, 2, 128, 16, BF)
    out, lse = same(kvd, c, "no groups")
    plain_lse = torch.empty_like(lse)
    plain = kvd.attend_paged(c.q, c.kc, c.vc, c.table, c.lens, lse=plain_lse)
    assert float((out.float() - plain.float()).abs().max()) <= 2.0 ** -7 * float(plain.abs().max())
    assert torch.isneginf(lse[1]).all() and bool((out[1] == 0).all())


def test_no_keys_at_all(kvd):
    c = Case([2], [0], [0, 5], 4, 2, 64, 16, F32)
    out, lse = same(kvd, c, "no keys")
    assert torch.isneginf(lse[0]).all() and bool((out[0] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_bad_groups(kvd, dtype):
    """group_lens that do not start at 0, fall or pass Q: no sequence has a prefix."""
    c = Case([2, 2], [70, 90], [9, 3, 30, 1], 8, 2, 64, 16, dtype)
    none = c.reference(prefix=False)
    for bad in ([1, 2, 4], [0, 3, 2], [0, 2, 5], [0, -1, 4], [-1, 2, 4]):
        c.glens = torch.tensor(bad, dtype=torch.int32, device="cuda")
        same(kvd, c, f"groups {bad}", ref=none, bits=kvd.DEV_SEQLENS)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_bad_prefixes(kvd, dtype):
    c = Case([1, 1], [70, 90], [9, 3], 8, 2, 64, 16, dtype)
    c.rows[0] = (c.rows[0][0][:0], c.rows[0][1][:0])
    none = c.reference()
    c.plens = torch.tensor([-1, 90], dtype=torch.int32, device="cuda")
    same(kvd, c, "negative", ref=none, bits=kvd.DEV_SEQLENS)
    c.plens = torch.tensor([c.ptable.shape[1] * 16 + 1, 90], dtype=torch.int32, device="cuda")
    same(kvd, c, "too long", ref=none, bits=kvd.DEV_TABLE_COLS)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("BS", [16, 128])
def test_dropped_pages(kvd, BS, dtype):
    """Blocks outside the cache, in a prefix and in a sequence: their tokens do not count."""
    c = Case([3], [5 * BS + 3], [2 * BS, 4, 1], 8, 2, 128, BS, dtype)
    c.ptable[0, 0], c.ptable[0, 3], c.ptable[0, 5] = -1, c.kc.shape[0], 2 ** 31 - 1
    c.table[0, 1] = -2
    ref = c.reference(drop=((0, 0), (0, 3), (0, 5), (1, 1)))
    same(kvd, c, "dropped", ref=ref, bits=kvd.DEV_BLOCK_RANGE)
    c.ptable[0, :] = -1
    ref = c.reference(drop=[(0, i) for i in range(6)] + [(1, 1)])
    same(kvd, c, "all dropped", ref=ref, bits=kvd.DEV_BLOCK_RANGE)


def test_bad_sequence_keeps_its_prefix(kvd):
    c = Case([3], [100], [20, 30, 10], 8, 2, 128, 16, BF)
    c.offset = torch.tensor([0, 3, 0], dtype=torch.int32, device="cuda")  # not a multiple of 16
    c.rows[2] = (c.rows[2][0][:0], c.rows[2][1][:0])
    same(kvd, c, "offset", ref=c.reference(), bits=kvd.DEV_SEQ_OFFSET)


def test_workspace_needs_no_zeros_and_is_used_again(kvd):
    """Garbage in the workspace, calls of other sizes one after the other, two streams."""
    cases = [Case([20], [900], [i % 5 for i in range(20)], 8, 2, 128, 16, BF, seed=1),
             Case([2, 1], [33, 400], [50, 0, 3], 16, 4, 64, 32, F32, seed=2),
             Case([1], [3000], [1], 32, 8, 128, 128, BF, seed=3)]
    need = max(kvd.attend_paged_prefix_workspace_bytes(
        c.q.shape[0], len(c.groups), c.Hq, c.Hkv, c.BS, c.ptable.shape[1], c.table.shape[1], c.D,
        c.dtype) for c in cases)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    first = [same(kvd, c, "first", workspace=ws)[0] for c in cases]
    side = torch.cuda.Stream()
    other = torch.full((need,), 1, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for c, want in zip(cases * 2, first * 2):
        with torch.cuda.stream(side):
            a = kvd.attend_paged_prefix(*c.args(), workspace=other)
        b = kvd.attend_paged_prefix(*c.args(), workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)  # to the bit: no order changes it


def test_graph(kvd):
    """Captured and replayed with other lengths, groups and pages behind the pointers."""
    a = Case([20, 5], [900, 77], [i % 5 for i in range(25)], 8, 2, 128, 16, BF, seed=1)
    b = Case([3, 22], [500, 901], [(i + 1) % 5 for i in range(25)], 8, 2, 128, 16, BF, seed=2)
    size = max(a.kc.shape[0], b.kc.shape[0])
    cols = max(a.ptable.shape[1], b.ptable.shape[1])

    def pad(t, n, dim):
        s = list(t.shape)
        s[dim] = n - s[dim]
        return torch.cat([t, torch.zeros(s, dtype=t.dtype, device="cuda")], dim)
    for c in (a, b):
        c.kc, c.vc, c.ptable = pad(c.kc, size, 0), pad(c.vc, size, 0), pad(c.ptable, cols, 1)
    static = [t.clone() for t in a.args()]
    kvd.attend_paged_prefix(*static)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lse = torch.empty(25, 8, device="cuda")
        out = kvd.attend_paged_prefix(*static, lse=lse)
    for c in (b, a, b):
        for t, x in zip(static, c.args()):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        lref.check("replayed", out, lse, *c.reference(), 910, BF)


def test_refusals(kvd):
    c = Case([2], [40], [5, 6], 8, 2, 64, 16, F32)
    q, kc, vc, pt, pl, gl, bt, sl = c.args()
    f = kvd.attend_paged_prefix
    for args, error in [((q.half(), kc, vc, pt, pl, gl, bt, sl), TypeError),
                        ((q, kc.to(BF), vc, pt, pl, gl, bt, sl), TypeError),
                        ((q, kc, vc[:1].contiguous(), pt, pl, gl, bt, sl), ValueError),
                        ((q, kc, vc, pt[0], pl, gl, bt, sl), ValueError),
                        ((q, kc, vc, pt.long(), pl, gl, bt, sl), TypeError),
                        ((q, kc, vc, pt, pl[:0], gl, bt, sl), ValueError),
                        ((q, kc, vc, pt, pl, gl[:1], bt, sl), ValueError),
                        ((q, kc, vc, pt, pl, gl, bt[:1], sl), ValueError),
                        ((q, kc, vc, pt, pl, gl, bt, sl[:2]), ValueError),
                        ((q[:, :3].contiguous(), kc, vc, pt, pl, gl, bt, sl), kvd.KvdError),
                        ((q.transpose(0, 1), kc, vc, pt, pl, gl, bt, sl), ValueError)]:
        with pytest.raises(error):
            f(*args)
    with pytest.raises(kvd.KvdError):
        f(*c.args(), workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        f(*c.args(), workspace=torch.zeros(1 << 24, dtype=torch.uint8))
