"""Attention of drafted tokens over the paged cache against binary64 on the
host: trees and chains, one token, every head layout and column count the
launch distinguishes, ragged lengths, both cache and query types, rows that see
nothing, pages that are not there, values that are not finite where a mask
hides them, rows that no request names, streams and graphs."""
import random

import pytest
import torch

import activation_sparse_mlp_amd as spffn
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, F8 = torch.float16, torch.float8_e4m3fn


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Problem:
    """A cache with requests of the given lengths and new tokens, on host and device."""

    def __init__(self, lens, news, heads, kv_heads, D, dtype, page, q_dtype, seed, spare=2,
                 behind=2, chain=False):
        rnd, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.lens, self.news, self.page, self.scale = lens, news, page, D ** -0.5
        self.heads, self.D = heads, D
        held = [-(-(t + n) // page) for t, n in zip(lens, news)]
        pages = sum(held) + spare
        ids = list(range(pages))
        rnd.shuffle(ids)
        self.table = torch.full((len(lens), max(max(held), 1) + 1), -1, dtype=torch.int32)
        for r, n in enumerate(held):
            for b in range(n):
                self.table[r, b] = ids.pop()
        k = torch.randn(pages * page, kv_heads, D, generator=g)
        v = torch.randn(pages * page, kv_heads, D, generator=g)
        k[:, :, 3] *= 6.0
        self.ks = self.vs = None
        if dtype == F8:
            self.ks = torch.rand(kv_heads, generator=g) * 0.05 + 0.02
            self.vs = torch.rand(kv_heads, generator=g) * 0.05 + 0.01
        self.k = ref.round_rows(k, dtype, self.ks)
        self.v = ref.round_rows(v, dtype, self.vs)
        self.starts = [0]
        for n in news:
            self.starts.append(self.starts[-1] + n)
        self.N = self.starts[-1] + behind
        bits = [b for n in news for b in ref.tree_bits(rnd, n)] + [0] * behind
        self.mask = None if chain else ref.as_int64(bits)
        self.q = (torch.randn(self.N, heads, D, generator=g) * 2.0).to(q_dtype)
        self.max_new = max(max(news), 1)
        self.pages = pages

    def cache(self):
        on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        return spffn.KVCache(ref.k_of_rows(self.k, self.pages, self.page).to(DEV),
                             ref.v_of_rows(self.v, self.pages, self.page).to(DEV), on(self.ks),
                             on(self.vs))

    def args(self):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        return dict(starts=i32(self.starts), lens=i32(self.lens), table=self.table.to(DEV),
                    mask=None if self.mask is None else self.mask.to(DEV), scale=self.scale,
                    max_new=self.max_new)

    def want(self, out0):
        return ref.attention(self.q, self.k, self.v, self.ks, self.vs, self.starts, self.lens,
                             self.table, self.page, self.mask, self.scale, self.max_new, out0,
                             self.q.dtype == F16)

    def check(self, any_odd=False):
        out0 = torch.full(self.q.shape, -3.0, dtype=self.q.dtype)
        out = out0.to(DEV)
        got = spffn.tree_attention(self.cache(), self.q.to(DEV), out=out, **self.args())
        torch.cuda.synchronize()
        assert got is out
        want, bound = self.want(out0)
        ref.close(got.cpu(), want, bound, any_odd)
        return got


CASES = [
    # lens, news, heads, kv_heads, D, page
    ([0], [1], 1, 1, 64, 16),                       # the first token of a request
    ([1], [1], 8, 8, 128, 16),
    ([31, 32, 33], [1, 1, 1], 8, 1, 128, 16),       # 8 columns
    ([5, 100, 0], [2, 1, 3], 3, 1, 96, 32),         # 9 columns at most
    ([64, 257], [4, 2], 8, 2, 128, 64),             # 16 columns
    ([70, 12, 300], [5, 1, 3], 10, 2, 64, 16),      # 25 columns
    ([200, 3], [11, 16], 8, 2, 128, 32),            # 64 columns
    ([129], [24], 15, 3, 64, 64),                   # 120 columns
    ([90, 17], [64, 7], 16, 2, 128, 128),           # 512 columns: several groups
    ([40, 0, 77], [0, 2, 1], 4, 2, 256, 16),        # a request without tokens
    ([77, 130], [9, 3], 12, 3, 256, 32),            # 36 columns of 256 dimensions
    ([500], [20], 16, 4, 256, 256),                 # 80 columns of 256 dimensions
    ([1500, 9, 640], [1, 1, 1], 32, 32, 64, 16),
    ([6000], [1], 16, 2, 128, 16),                  # one request over many workgroups
    ([3000, 1], [40, 3], 12, 1, 96, 64),
]


@pytest.mark.parametrize("q_dtype", [torch.float32, F16])
@pytest.mark.parametrize("dtype", [F16, F8])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_trees(case, dtype, q_dtype):
    lens, news, heads, kv, D, page = CASES[case]
    Problem(lens, news, heads, kv, D, dtype, page, q_dtype, seed=case).check()


@pytest.mark.parametrize("dtype", [F16, F8])
def test_chain_without_a_mask(dtype):
    Problem([0, 50, 127], [7, 64, 1], 8, 4, 128, dtype, 16, torch.float32, seed=40,
            chain=True).check()


def test_many_requests():
    rnd = random.Random(5)
    lens = [rnd.choice([0, 1, 17, 40, 90]) for _ in range(150)]
    news = [rnd.choice([0, 1, 1, 2]) for _ in range(150)]
    Problem(lens, news, 4, 2, 64, F16, 16, torch.float32, seed=41).check()


@pytest.mark.parametrize("dtype", [F16, F8])
@pytest.mark.parametrize("news", [1, 5, 20])
def test_rows_that_see_nothing(dtype, news):
    p = Problem([0, 40, 0], [news] * 3, 8, 1, 128, dtype, 16, torch.float32, seed=42)
    p.mask[::2] = 0          # in the first and last request these rows have no key at all
    got = p.check()
    assert bool((got[0] == 0).all())


@pytest.mark.parametrize("news", [1, 3, 20])
def test_unmapped_and_bad_pages(news):
    p = Problem([100, 64, 40], [news] * 3, 8, 2, 64, F16, 16, torch.float32, seed=43)
    p.table[0, 2] = -1
    p.table[0, 4] = p.pages
    p.table[1, :] = -1       # nothing of this request is there
    p.table[2, 0] = 2 ** 31 - 1
    p.check()


def test_lengths_past_the_table_and_tokens_past_max_new():
    p = Problem([30, 47], [4, 6], 4, 2, 64, F16, 16, torch.float32, seed=44)
    p.table = p.table[:, :3].contiguous()   # 48 tokens: the second request has room for one
    p.lens[0] = 200                          # more than the row holds: all of it is seen
    p.max_new = 5
    p.check()
    p.lens[0] = -4                           # as none
    p.check()


@pytest.mark.parametrize("dtype", [F16, F8])
@pytest.mark.parametrize("q_dtype", [torch.float32, F16])
@pytest.mark.parametrize("news,heads", [(3, 4), (4, 16), (24, 8)])
def test_not_finite_where_hidden(dtype, q_dtype, news, heads):
    p = Problem([45, 20], [news, news], heads, 2, 64, dtype, 16, q_dtype, seed=45)
    slot = lambda r, t: int(p.table[r, t // 16]) * 16 + t % 16  # noqa: E731
    bad = [float("nan")] if dtype == F8 else [float("nan"), float("inf"), float("-inf")]
    # a drafted token of request 0 holds them, and only itself and its heirs may see them
    for i, b in enumerate(bad):
        p.v[slot(0, 46), 0, 5 + i] = b
    p.k[slot(0, 47), 1, 2] = float("nan")
    # memory behind each request's last token
    for r, t in ((0, 45 + news), (1, 20 + news)):
        if t % 16:
            p.k[slot(r, t)] = float("nan")
            p.v[slot(r, t)] = float("nan")
    p.check()


@pytest.mark.parametrize("q_dtype", [torch.float32, F16])
def test_not_finite_where_seen(q_dtype):
    p = Problem([45, 80, 33], [3, 2, 1], 4, 2, 64, F16, 16, q_dtype, seed=46)
    slot = lambda r, t: int(p.table[r, t // 16]) * 16 + t % 16  # noqa: E731
    p.v[slot(1, 7), 0, 9] = float("nan")
    p.v[slot(1, 70), 1, 1] = float("inf")
    p.v[slot(2, 32), 0, 0] = float("-inf")
    p.q[0, 1, 4] = float("inf")
    p.q[1, 2, 4] = float("nan")
    p.check(any_odd=True)


def test_infinite_keys():
    # fp16 queries: as the formula has it
    p = Problem([20, 1, 40], [1, 1, 1], 2, 1, 64, F16, 16, F16, seed=47)
    slot = lambda r, t: int(p.table[r, t // 16]) * 16 + t % 16  # noqa: E731
    p.q[:] = p.q.abs() + 0.1
    p.k[slot(0, 3), 0, 5] = float("-inf")     # a score of -inf: a weight of 0
    p.k[slot(1, 0), 0, 5] = float("-inf")     # every score -inf: NaN
    p.k[slot(1, 1), 0, 5] = float("-inf")
    p.k[slot(2, 30), 0, 5] = float("inf")     # a score of +inf: NaN
    got = p.check()
    assert bool(torch.isfinite(got[0]).all()) and bool(torch.isnan(got[1:3]).all())


@pytest.mark.parametrize("heads", [2, 6, 40])
def test_infinite_keys_of_split_queries(heads):
    # fp32 queries: NaN for the tokens that see such a key (or, where its score is
    # -inf in both halves, a weight of 0), the others as ever
    p = Problem([20, 40], [2, 1], heads, 1, 64, F16, 16, torch.float32, seed=53)
    p.mask[:3] = ref.as_int64([1, 2, 1])
    slot = lambda r, t: int(p.table[r, t // 16]) * 16 + t % 16  # noqa: E731
    out0 = torch.full(p.q.shape, -3.0)
    want, bound = p.want(out0)
    p.k[slot(0, 21), 0, 5] = float("inf")     # seen by token 1 alone
    got = spffn.tree_attention(p.cache(), p.q.to(DEV), out=out0.to(DEV), **p.args()).cpu()
    keep = torch.arange(p.N) != 1
    ref.close(got[keep], want[keep], bound[keep])
    nan = torch.isnan(got[1])
    assert bool((nan.all(-1) | ~nan.any(-1)).all()) and bool(nan.any())


@pytest.mark.parametrize("news", [1, 6])
def test_scales_of_queries(news):
    p = Problem([100, 33], [news, news], 4, 1, 64, F16, 16, torch.float32, seed=48)
    p.q[0] *= 1e-30
    p.q[1] *= 300.0          # weights down to e^-1000s
    p.q[p.starts[1], 0] = 0.0
    p.check()
    p.scale = -0.3
    p.check()
    p.scale = 0.0
    p.check()


def test_far_apart_scores_raise_the_running_maximum():
    p = Problem([2000], [1], 4, 4, 64, F16, 16, torch.float32, seed=49)
    ramp = torch.linspace(-60, 60, p.k.shape[0])
    order = [int(p.table[0, t // 16]) * 16 + t % 16 for t in range(2001)]
    for i, s in enumerate(order):
        p.k[s, :, 0] = ramp[i]
    p.q[:, :, 0] = 6.0
    p.check()


def test_strided_rows_and_streams():
    p = Problem([60, 9], [3, 2], 8, 4, 128, F16, 32, torch.float32, seed=50)
    out0 = torch.full(p.q.shape, -3.0)
    want, bound = p.want(out0)
    qkv = torch.randn(p.N, 16, 128, device=DEV)
    qkv[:, :8] = p.q.to(DEV)
    wide = torch.full((p.N, 11, 128), -3.0, device=DEV)
    cache, args = p.cache(), p.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = spffn.tree_attention(cache, qkv[:, :8], out=wide[:, 2:10], **args)
    s.synchronize()
    ref.close(got.cpu(), want, bound)
    assert bool((wide[:, :2] == -3).all()) and bool((wide[:, 10:] == -3).all())


def test_repeats_bitwise_and_graph():
    p = Problem([900, 30, 411], [5, 2, 1], 8, 2, 128, F16, 16, torch.float32, seed=51)
    cache, args = p.cache(), p.args()
    q = p.q.to(DEV)
    ws = cache.workspace(8, p.max_new)
    out = torch.zeros_like(q)
    first = spffn.tree_attention(cache, q, out=out, ws=ws, **args).clone()
    ws.fill_(255)            # what the workspace holds does not matter
    assert torch.equal(spffn.tree_attention(cache, q, out=out, ws=ws, **args), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spffn.tree_attention(cache, q, out=out, ws=ws, **args)
    g = torch.Generator().manual_seed(1)
    for i, lens in enumerate(([900, 30, 411], [3, 0, 411], [0, 31, 7], [896, 2, 100])):
        q.copy_(torch.randn(q.shape, generator=g))
        args["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        want = spffn.tree_attention(cache, q, out=torch.zeros_like(q), **args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_far_offsets():
    # a cache past 2^32 bytes and 2^31 elements, the request's pages at its end
    H, D, page, L = 8, 128, 64, 200
    pages = (1 << 31) // (H * D * page) + 5
    k = torch.zeros(pages, H, D // 8, page, 8, dtype=F16, device=DEV)
    v = torch.zeros(pages, H, page // 8, D, 8, dtype=F16, device=DEV)
    small = Problem([L], [2], 16, H, D, F16, page, torch.float32, seed=52, spare=0)
    n = small.pages
    k[-n:] = ref.k_of_rows(small.k, n, page).to(DEV)
    v[-n:] = ref.v_of_rows(small.v, n, page).to(DEV)
    out0 = torch.full(small.q.shape, -3.0)
    want, bound = small.want(out0)
    args = small.args()
    args["table"] = torch.where(args["table"] >= 0, args["table"] + pages - n, args["table"])
    got = spffn.tree_attention(spffn.KVCache(k, v), small.q.to(DEV), out=out0.to(DEV), **args)
    ref.close(got.cpu(), want, bound)
