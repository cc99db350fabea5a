"""Attention over shared and own tokens on the GPU, against attention over both in a row in 64 bits."""

import math
import re

import pytest
import torch

import bit_matmul_amd as bm
from tests import attn_util as U

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


class Groups(U.Sequences):
    """Groups of sequences. groups: (shared tokens, [(queries, own tokens), ...]) of each; shared tokens of None:
    sequences of no group."""

    wider = 0   # of the bound of the own tokens, more than there are

    def __init__(self, groups, *, q_heads, kv_heads, head_dim, group, page, dtype, seed=0, spare=2, counted=False):
        g = torch.Generator().manual_seed(seed)
        self.page, self.group, self.dtype = page, group, dtype
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.own = [s for _, seqs in groups for s in seqs]
        self.prefix_of, self.shared, cu_groups, at = [], [], [0], 0
        for n, seqs in groups:
            self.prefix_of += [-1 if n is None else len(self.shared)] * len(seqs)
            at += len(seqs)
            if n is None:
                assert not self.shared   # those come first
                cu_groups = [at]
            else:
                self.shared.append(n)
                cu_groups.append(at)
        self.lens = [(q, n + (self.shared[p] if p >= 0 else 0)) for (q, n), p in zip(self.own, self.prefix_of)]
        need = [-(-n // page) for n in self.shared] + [-(-n // page) for _, n in self.own]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.spare = order[sum(need):]
        tables = torch.zeros(len(need), max(need + [1]), dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            tables[i, :n] = order[at:at + n]
            at += n
        G = len(self.shared)
        self.prefix_table = tables[:G, :max(need[:G] + [1])].contiguous()
        self.page_table = tables[G:, :max(need[G:] + [1])].contiguous()
        shape = (pages, kv_heads, page, head_dim)
        self.sides = []
        for _ in range(2):
            x = torch.randn(shape, generator=g)
            x[..., ::16] *= 3
            self.sides.append(U.quantise(x.to(BF), group))
        total = sum(q for q, _ in self.own)
        self.q = (1.5 * torch.randn(total, q_heads, head_dim, generator=g)).to(dtype)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)
        self.cu = i32([0] + [sum(q for q, _ in self.own[:i + 1]) for i in range(len(self.own))])
        self.kv_lens, self.prefix_lens, self.cu_groups = i32([n for _, n in self.own]), i32(self.shared), i32(cu_groups)
        if counted:
            self.count()

    def places(self, b, kv):
        """(page, slot) of a sequence's tokens, the shared ones first."""
        p = self.prefix_of[b]
        n = min(kv, self.shared[p]) if p >= 0 else 0
        j, i = torch.arange(n), torch.arange(kv - n)
        page = torch.cat([self.prefix_table[p].long()[j // self.page] if n else j, self.page_table[b].long()[i // self.page]])
        return page, torch.cat([j % self.page, i % self.page])

    def tokens(self, side, b, kv):
        codes, scale, bias = self.sides[side]
        page, off = self.places(b, kv)
        return (U.values(codes[page, :, off], scale[page, :, off], bias[page, :, off]),
                U.centre(scale[page, :, off], bias[page, :, off], self.group))

    def count(self):
        """Queries of zero, and values that are 1 in dim j / 32 + 7 head for a sequence's token j and 0 elsewhere: outputs
        count tokens, and the lse all of them."""
        pages = self.sides[0][0].shape[0]
        ones = torch.ones(pages, self.kv_heads, self.page, self.head_dim // self.group, dtype=torch.float64)
        values = torch.full((pages, self.kv_heads, self.page, self.head_dim), 9)
        for b, (_, kv) in enumerate(self.lens):
            page, off = self.places(b, kv)
            j = torch.arange(kv)
            for h in range(self.kv_heads):
                values[page, h, off] = 0
                values[page, h, off, (j // 32 + 7 * h) % self.head_dim] = 1
        self.sides = [(self.sides[0][0], ones, 0 * ones), (values, ones, 0 * ones)]
        self.q = torch.zeros_like(self.q)

    def bounds(self):
        of_group = [sum(q for (q, _), p in zip(self.own, self.prefix_of) if p == g) for g in range(len(self.shared))]
        return dict(max_group_q=max(of_group + [0]), max_prefix=max(self.shared + [0]),
                    max_q=max(q for q, _ in self.own), max_kv=max(n for _, n in self.own) + self.wider)

    def run(self, cache=None, q=None, **kw):
        """(out, lse, status word)"""
        q = self.q.cuda() if q is None else q
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        there = [t.cuda() for t in (self.prefix_table, self.prefix_lens, self.cu_groups, self.page_table, self.kv_lens, self.cu)]
        out = bm.kv_attention_shared(q, self.cache("cuda") if cache is None else cache, *there, lse=lse, status=status,
                                     **{**self.bounds(), **kw})
        return out.cpu().double(), lse.cpu().double(), status.item()


def check(s, out_dtype, scale=None, **kw):
    scale = 1 / math.sqrt(s.head_dim) if scale is None else scale
    out, lse, status = s.run(out_dtype=out_dtype, scale=scale, **kw)
    want, want_lse, tol, tol_lse = s.reference(out_dtype, scale)
    assert status == 0
    assert ((out - want).abs() <= tol).all()
    same = (lse == want_lse) | ((lse - want_lse).abs() <= tol_lse)
    assert same.all()


def beams(n, q, own):
    return [(q, own)] * n


CASES = {  # groups, query heads, kv heads, dims, group, page, type, type of the output
    "one beam": ([(100, beams(1, 1, 7))], 4, 1, 64, 32, 16, BF, BF),
    "four beams": ([(573, beams(4, 1, 29))], 40, 8, 128, 64, 64, BF, BF),
    "ragged groups": ([(700, beams(4, 1, 33)), (3, beams(3, 1, 80)), (1200, beams(2, 1, 1)), (64, beams(1, 1, 64))], 10, 2, 128, 32, 16, F16, F32),
    "nothing of its own": ([(90, [(1, 0), (1, 0)]), (40, [(1, 0)])], 8, 2, 64, 64, 32, BF, F32),
    "nothing shared": ([(0, [(1, 50), (2, 60)]), (0, [(1, 1)])], 8, 2, 64, 64, 32, BF, F32),
    "nothing at all": ([(0, [(1, 0), (1, 5)]), (17, [(1, 0)])], 6, 2, 128, 128, 16, BF, F32),
    "no group": ([(None, [(1, 40), (3, 30)]), (100, [(1, 20)])], 6, 2, 128, 64, 64, F16, F32),
    "no groups": ([(None, [(1, 40), (3, 30), (0, 4)])], 6, 2, 128, 64, 64, F16, F16),
    "idle sequences": ([(100, [(0, 5), (1, 9), (0, 0), (2, 4)]), (50, []), (60, [(0, 3)]), (70, [(1, 1)])], 4, 4, 64, 32, 16, BF, F32),
    "guesses": ([(333, [(5, 9), (2, 30), (1, 1), (4, 4)])], 16, 2, 256, 32, 16, F16, F32),
    "many beams": ([(2000, beams(40, 1, 12))], 10, 2, 128, 64, 64, BF, F32),
    "many rows, split": ([(5000, beams(32, 1, 50))], 40, 8, 128, 64, 32, BF, F32),
    "many rows, narrow": ([(3000, beams(48, 1, 20)), (2500, beams(30, 1, 9))], 16, 2, 64, 32, 16, F16, F32),
    "many rows, wide": ([(2100, beams(40, 1, 17))], 8, 1, 256, 64, 64, BF, BF),
    "long own tokens": ([(900, [(1, 3000), (1, 40), (1, 1500)]), (100, [(1, 700)])], 8, 2, 128, 64, 64, BF, F32),
    "100 sequences": ([(200, beams(50, 1, 31)), (333, beams(50, 1, 65))], 3, 3, 64, 64, 64, F16, F16),
    "chunks": ([(600, [(100, 100), (77, 200), (301, 301)]), (70, [(30, 30)])], 8, 2, 128, 64, 64, BF, BF),
    "chunks, binary16": ([(1500, [(150, 150), (90, 333)])], 10, 2, 64, 32, 16, F16, F32),
    "chunks, wide": ([(130, [(90, 90), (200, 290)])], 4, 1, 256, 128, 32, F16, F16),
    "share of 64": ([(100, [(1, 20), (2, 9)])], 64, 1, 64, 64, 16, BF, F32),
    "equal heads": ([(1000, beams(3, 1, 40))], 5, 5, 128, 128, 256, F16, F32),
}


# Bounds decide which kernels run: small cases go through one launch as they are, through a pass over the shared
# tokens and one over the own ones with a wide bound of the former, and with a wide bound of the latter through a join.
WIDE = {"as they are": {}, "wide": dict(max_prefix=100000), "wide own": dict(max_prefix=3000, max_kv=50000)}


@pytest.mark.parametrize("bounds", WIDE)
@pytest.mark.parametrize("name", CASES)
def test_against_64_bits(name, bounds):
    groups, hq, hk, D, group, page, dtype, out_dtype = CASES[name]
    s = Groups(groups, q_heads=hq, kv_heads=hk, head_dim=D, group=group, page=page, dtype=dtype, seed=len(name))
    check(s, out_dtype, **{k: max(v, s.bounds()[k]) for k, v in WIDE[bounds].items()})


def test_what_runs():
    """Each of the forms above is taken: by the names of the kernels of a call."""
    kw = dict(q_heads=40, kv_heads=8, head_dim=128, group=64, page=64, dtype=BF)
    small, many = Groups([(573, beams(4, 1, 29))], **kw), Groups([(2000, beams(64, 1, 29)), (10, [(70, 70)])], **kw)

    def names(s, **bounds):
        s.run(**bounds)
        return [re.sub(r"<([^>]*)>.*", lambda m: " " + m[1].split(", ")[-1], line) for line in bm.bitmm_last_launches()]

    assert names(small) == ["attention_rows_kernel both"]
    assert names(small, max_prefix=1281) == ["attention_rows_kernel prefix", "attention_rows_kernel own"]
    assert names(small, max_kv=20000) == ["attention_rows_kernel prefix", "attention_rows_kernel own", "attention_join_shared_kernel 128"]
    assert names(many) == ["attention_tiles_kernel prefix", "attention_tiles_kernel own"]
    chunk = Groups([(600, [(400, 400)])], **kw)
    assert names(chunk, max_kv=20000)[1:] == ["attention_tiles_kernel own", "attention_join_shared_kernel 128"]


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    check(Groups([(130, beams(3, 1, 40))], q_heads=8, kv_heads=2, head_dim=64, group=32, page=16, dtype=BF, seed=1), F32, scale)


COUNTED = {
    "long": ([(40000, beams(4, 1, 300))], 8, 2, 128),
    "long, many rows": ([(33000, beams(64, 1, 77))], 10, 2, 128),
    "many rows, 64 dims": ([(9001, beams(33, 1, 1000)), (20000, beams(20, 1, 5))], 8, 1, 64),
    "wide": ([(17000, beams(30, 1, 500))], 16, 2, 256),
    "chunks": ([(7000, [(300, 300), (200, 2500), (1, 1)])], 4, 1, 64),
    "own longer": ([(500, [(1, 20000), (1, 3), (1, 9000)])], 8, 1, 128),
}


@pytest.mark.parametrize("name", COUNTED)
def test_every_token_counts_once(name):
    """Sums of whole numbers below 2^24 times powers of two are exact in f32, and so are 2^0 weights between parts:
    outputs are a division and a product away (4 half steps), the lse of up to 16 two of its steps."""
    groups, hq, hk, D = COUNTED[name]
    s = Groups(groups, q_heads=hq, kv_heads=hk, head_dim=D, group=64, page=64, dtype=BF, counted=True)
    out, lse, status = s.run(out_dtype=F32)
    assert status == 0
    for b, (nq, kv) in enumerate(s.lens):
        seen = torch.arange(kv - nq, kv) + 1
        runs = (seen[:, None] - 32 * torch.arange(-(-kv // 32))).clamp(0, 32).double()
        for head in range(hq):
            h = head * hk // hq
            want = torch.zeros(nq, D, dtype=torch.float64)
            want.index_add_(1, (torch.arange(runs.shape[1]) + 7 * h) % D, runs)
            want /= seen[:, None]
            at = slice(int(s.cu[b]), int(s.cu[b + 1]))
            assert ((out[at, head] - want).abs() <= 4 * 2.0 ** -24 * want).all()
            assert ((lse[at, head] - seen.double().log()).abs() <= 2.0 ** -18).all()


@pytest.mark.parametrize("wide", [0, 2000])
def test_queries_before_their_own_tokens(wide):
    """They see all that is shared, like a query with no tokens of its own."""
    kw = dict(q_heads=4, kv_heads=2, head_dim=64, group=32, page=16, dtype=BF, seed=3)
    s = Groups([(50, [(3, 1)])], **kw)
    s.wider = wide
    out, lse, status = s.run(out_dtype=F32)
    alone = Groups([(50, [(1, 0), (1, 0), (1, 1)])], **kw)
    alone.sides, alone.q, alone.prefix_table = s.sides, s.q, s.prefix_table
    alone.page_table = s.page_table.expand(3, -1).contiguous()
    want, want_lse, tol, tol_lse = alone.reference(F32, 1 / 8)
    assert status == 0 and ((out - want).abs() <= tol).all() and ((lse - want_lse).abs() <= tol_lse).all()


def test_strides_and_rows_of_no_sequence():
    """Slices of a fused projection, and rows behind the last sequence, which stay as they are."""
    s = Groups([(300, beams(3, 1, 20)), (40, beams(2, 2, 9))], q_heads=6, kv_heads=2, head_dim=64, group=32, page=16, dtype=BF, seed=4)
    T = s.q.shape[0]
    wide = torch.randn(T + 3, 11, 64).to(BF).cuda()
    wide[:T, 2:8] = s.q.cuda()
    whole = torch.full((T + 3, 9, 64), 5.0, dtype=BF, device="cuda")
    there = [t.cuda() for t in (s.prefix_table, s.prefix_lens, s.cu_groups, s.page_table, s.kv_lens, s.cu)]
    b = s.bounds()
    need = bm.bitmm_kv_attention_shared_workspace_bytes(T + 3, 5, 2, *b.values(), 6, 2, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    lse = torch.full((T + 3, 6), 9.0, device="cuda")
    bm.bitmm_kv_attention_shared(wide[:, 2:8], s.cache("cuda"), *there, whole[:, 1:7], ws, lse=lse, **b)
    want, want_lse, _ = s.run()
    assert torch.equal(whole[:T, 1:7].cpu().double(), want) and torch.equal(lse[:T].cpu().double(), want_lse)
    assert (whole[T:] == 5).all() and (whole[:, 0] == 5).all() and (whole[:, 7:] == 5).all() and (lse[T:] == 9).all()


@pytest.mark.parametrize("wide", [0, 2000])
@pytest.mark.parametrize("rows", [1, 40])
def test_out_of_range(rows, wide):
    """What passes the bounds is cut and reported; pages outside the cache are seen by nobody. wide: more of a bound of
    the own tokens, for the kernels of two passes."""
    kw = dict(q_heads=8, kv_heads=2, head_dim=64, group=32, page=16, dtype=BF)
    groups = [(200, beams(rows, 1, 20)), (90, beams(rows, 1, 20))]
    s = Groups(groups, seed=5, **kw)
    s.wider = wide
    full, _, ok = s.run()
    assert ok == 0
    n = rows * 1
    # a prefix longer than the bound: as if it were that long
    out, _, status = s.run(max_prefix=90)
    short = Groups([(90, groups[0][1]), groups[1]], seed=5, **kw)
    short.wider = wide
    short.sides, short.q, short.page_table = s.sides, s.q, s.page_table
    short.prefix_table = s.prefix_table[:, :6].contiguous()
    assert status == 1 and torch.equal(out, short.run()[0])
    # a bad page among the shared tokens of the second group, and among the own ones of its first sequence
    for table, at in ((s.prefix_table, (1, 2)), (s.page_table, (rows, 1))):
        for bad in (-1, s.sides[0][0].shape[0], 2 ** 31 - 1, -2 ** 31):
            was = table[at].item()
            table[at] = bad
            out, lse, status = s.run(out_dtype=F32)
            table[at] = was   # the tokens that are lost, by the page they had
            first = 32 if table is s.prefix_table else 90 + 16
            hide = lambda b, j: ((j >= first) & (j < first + 16)) if (b >= rows if first == 32 else b == rows) else j < 0
            want, want_lse, tol, tol_lse = s.reference(F32, 1 / 8, hide=hide)
            assert status == 1 and ((out - want).abs() <= tol).all() and ((lse - want_lse).abs() <= tol_lse).all()
    # groups that name sequences which are not there, and lengths that are negative
    for cu in ([0, rows, 2 * rows + 1], [-1, rows, 2 * rows]):
        s.cu_groups = torch.tensor(cu, dtype=torch.int32)
        out, _, status = s.run(**short.bounds() | dict(max_prefix=200))
        assert status == 1 and torch.equal(out, full)
    s.cu_groups = torch.tensor([0, rows, 2 * rows], dtype=torch.int32)
    s.prefix_lens[0] = -4
    out, _, status = s.run(max_prefix=200)
    assert status == 1 and torch.equal(out[n:], full[n:])
    s.prefix_lens[0] = 200
    # more queries in a group than its bound: rows past it are not written
    if rows > 1:
        q = s.q.cuda()
        there = [t.cuda() for t in (s.prefix_table, s.prefix_lens, s.cu_groups, s.page_table, s.kv_lens, s.cu)]
        b = {**s.bounds(), "max_group_q": 7}
        ws = torch.empty(bm.bitmm_kv_attention_shared_workspace_bytes(2 * n, 2 * rows, 2, *b.values(), 8, 2, 64), dtype=torch.uint8, device="cuda")
        out, word = torch.full_like(q, 3.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        bm.bitmm_kv_attention_shared(q, s.cache("cuda"), *there, out, ws, status=word, **b)
        out = out.cpu().double()
        assert word.item() == 1
        for g in range(2):
            assert (out[g * n + 7:(g + 1) * n] == 3).all()
            near = out[g * n:g * n + 7] - full[g * n:g * n + 7]   # other splits, another order of sums
            assert near.abs().max() <= 2.0 ** -7 * full.abs().max()


@pytest.mark.parametrize("wide", [0, 2000])
@pytest.mark.parametrize("rows", [2, 40])
def test_what_is_not_finite(rows, wide):
    """A token whose scale is not finite makes NaN of the rows that see it, and slots that hold no token may hold anything."""
    s = Groups([(70, beams(rows, 1, 20)), (40, beams(rows, 1, 9))], q_heads=8, kv_heads=2, head_dim=128, group=64, page=16, dtype=BF, seed=6)
    s.wider = wide
    clean, _, _ = s.run()
    page = s.prefix_table[0, 4].item()          # slots 6 and on of this page hold no token
    s.sides[0][1][page, :, 6:] = math.nan
    s.sides[1][2][page, :, 6:] = math.inf
    own = s.page_table[0, 1].item()
    s.sides[0][2][own, :, 4:] = math.nan
    out, _, status = s.run()
    assert status == 0 and torch.equal(out, clean)
    s.sides[0][1][page, 1, 5] = math.inf        # a shared token, second kv head
    out, _, _ = s.run()
    assert out[:rows, 4:].isnan().all() and torch.equal(out[:rows, :4], clean[:rows, :4]) and torch.equal(out[rows:], clean[rows:])


@pytest.mark.parametrize("rows", [3, 33])
def test_captured_on_another_stream(rows):
    """Replays over growing sequences, with a workspace that others write to between them."""
    s = Groups([(600, beams(rows, 1, 90)), (450, beams(rows, 1, 90))], q_heads=10, kv_heads=2, head_dim=128, group=64, page=32, dtype=BF, seed=7)
    cache, q = s.cache("cuda"), s.q.cuda()
    there = [t.cuda() for t in (s.prefix_table, s.prefix_lens, s.cu_groups, s.page_table, s.kv_lens, s.cu)]
    b = s.bounds()
    ws = torch.empty(bm.bitmm_kv_attention_shared_workspace_bytes(2 * rows, 2 * rows, 2, *b.values(), 10, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    call = lambda to, stream=None: bm.bitmm_kv_attention_shared(q, cache, *there, to, ws, stream=stream, **b)
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for i, n in enumerate((1, 40, 64, 90)):
        there[4].fill_(n)
        there[1][0] = 600 - 100 * i
        q.copy_(torch.randn_like(q, dtype=F32).to(BF))
        ws.fill_(0xFF if i % 2 else 0)
        graph.replay()
        torch.cuda.synchronize()
        replayed, eager = out.clone(), torch.empty_like(out)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        call(eager, stream)
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(replayed, eager) and replayed.isfinite().all()
    s.kv_lens.fill_(90)
    s.prefix_lens[0] = 300
    s.shared[0] = 300
    s.lens = [(qn, n + s.shared[p]) for (qn, n), p in zip(s.own, s.prefix_of)]
    s.q = q.cpu()
    want, _, tol, _ = s.reference(BF, 1 / math.sqrt(128))
    assert ((replayed.cpu().double() - want).abs() <= tol).all()


def test_pages_past_32_bits():
    """Codes more than 2^32 bytes into the cache are written, seen and copied like those of a small one."""
    pages, far, page, D = 140, 139860, 256, 256
    small, large = (bm.KVCache.empty(n, page, 1, D, 128) for n in (pages, far + pages))
    assert large.k_codes.numel() * 4 > 2 ** 32 + 140 * page * 128
    g = torch.Generator().manual_seed(9)
    T, beams_n = 1500, 3
    k, v = (torch.randn(T, 1, D, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(beams_n, 4, D, generator=g).to(BF).cuda()
    freq, _ = bm.rope_frequencies(D, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    outs = []
    for cache, base in ((small, 0), (large, far)):
        order = torch.arange(6, device="cuda") * 20 + base + 3    # scattered pages, the last near the end
        at = torch.arange(T, device="cuda")
        bm.bitmm_qk_norm_rope_append(None, k, v, None, None, pos, freq, None, order[at // page] * page + at % page, cache)
        table = (order[5:].int().expand(3) + torch.zeros(3, dtype=torch.int32, device="cuda"))[:, None].contiguous()
        table, lens, slots = bm.kv_beam_reorder(bm.KVLayers([cache]), table, i32([200, 200, 200]), i32([[0, 1, 2]]), first_page=base + 100,
                                                pages_per_group=40)
        bm.bitmm_kv_append(k[:3], v[:3], slots, cache)
        outs.append([table - base, slots - base * page] + [
            bm.kv_attention_shared(q, cache, order[:5][None].int(), i32([1280]), i32([0, 3]), table, lens, i32([0, 1, 2, 3]),
                                   max_group_q=3, max_prefix=bound, max_q=1, max_kv=201) for bound in (1024, 1280, 5000)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert outs[0][-1].isfinite().all()
