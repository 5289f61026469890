"""The attention half together with the sparse FFN, as a decode loop uses them:
block tables, then for every layer attn_step and a one-layer decode_step on the
same residual stream, for several steps with drafted tokens, requests that end
and a padded batch; against binary64 on the host, and captured into a graph."""
import random

import numpy as np
import pytest
import torch

import activation_sparse_mlp_amd as spffn
import oracle
from tests import attn_ref as ref
from tests.gpu_helpers import gpu_layer, np_layer
from workloads import TINY, make_layer

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-5


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Stack:
    """Layers of width TINY.d: 8 query and 2 kv heads of 64, then the TINY sparse FFN."""

    def __init__(self, layers, dtype, seed, pages=40, page=16):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv, self.D, self.d, self.page = 8, 2, 64, TINY.d, page
        self.host, self.attn, self.cache, self.ffn, self.np_ffn = [], [], [], [], []
        for l in range(layers):
            ws = []
            for rows, cols, group in (((8 + 4) * 64, self.d, 32), (self.d, 512, 128)):
                codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g)
                sc = (torch.rand(rows, cols // group, generator=g) * 0.02 + 0.005).half()
                z = torch.randint(5, 11, sc.shape, dtype=torch.uint8, generator=g)
                ws.append((spffn.Q4Matrix(codes.to(DEV), sc.to(DEV), z.to(DEV), group=group),
                           ref.q4_weights(codes, sc, z, group)))
            bias = torch.randn(12 * 64, generator=g) * 0.1
            self.attn.append(spffn.Attention(ws[0][0], ws[1][0], 8, 64, qkv_bias=bias.to(DEV),
                                             rms_eps=EPS))
            self.host.append((ws[0][1], ws[1][1], bias))
            E = ref.packet(dtype)
            scale = None if E == 8 else torch.tensor([0.02, 0.03])
            dev = None if scale is None else scale.to(DEV)
            k = torch.zeros(pages, 2, 64 // E, page, E).to(dtype).to(DEV)
            v = torch.zeros(pages, 2, page // E, 64, E).to(dtype).to(DEV)
            self.cache.append((spffn.KVCache(k, v, dev, dev), scale))
            w = make_layer(TINY, l, seed=seed)
            self.ffn.append(spffn.Model([gpu_layer(w)], rms_eps=EPS))
            self.np_ffn.append(np_layer(w))

    def step(self, x, lens, adds, table, free, n_free, n, mask, max_new):
        t = spffn.block_tables(lens, adds, table, free, n_free, self.page, n)
        h = x.clone()
        for attn, (cache, _), ffn in zip(self.attn, self.cache, self.ffn):
            spffn.attn_step(attn, cache, h, t["starts"], lens, t["slots"], table, mask=mask,
                            max_new=max_new, h=h)
            spffn.decode_step(ffn, h, h=h)
        return h, t


def host_layer(s, l, x, rows, starts, lens, slots, table, mask, max_new):
    """One layer on the host: x [B, d] float64; rows, the cache's (k, v) rows after the GPU's
    call, are what attention reads.  They have to hold the new keys and values as one rounding
    of a value within the matvec's bound of the host's: half a step of the type, relative, or
    half its smallest subnormal, beyond that bound."""
    wqkv, wout, bias = s.host[l]
    B, scale = x.shape[0], s.cache[l][1]
    split = lambda t: t.view(B, 12, 64).split([8, 2, 2], 1)  # noqa: E731
    y, bound = ref.q4_matvec(wqkv, x, bias, rms_eps=EPS)
    (q, *new), (_, *bounds) = split(y), split(bound)
    f8 = rows[0].dtype != torch.float16
    half, least = (2.0 ** -4, 2.0 ** -10) if f8 else (2.0 ** -11, 2.0 ** -25)
    for got, want, far in zip(rows, new, bounds):
        unit = scale.double().view(2, 1) if f8 else torch.ones(2, 1, dtype=torch.float64)
        if f8:
            want = torch.minimum(torch.maximum(want, -448 * unit), 448 * unit)
        for b, slot in enumerate(slots):
            if slot >= 0:
                err = (got[slot].double() * unit - want[b]).abs()
                assert (err <= far[b] + half * (want[b].abs() + far[b]) + least * unit).all()
    o, _ = ref.attention(q, rows[0], rows[1], scale, scale, starts, lens, table, s.page, mask,
                         64 ** -0.5, max_new, torch.zeros(B, 8, 64), False)
    return x + ref.q4_matvec(wout, o.reshape(B, 512))[0]


@pytest.mark.parametrize("dtype", [torch.float16, torch.float8_e4m3fn])
def test_steps_of_attention_and_sparse_ffn(dtype):
    layers, page = 2, 16
    s = Stack(layers, dtype, seed=11)
    rnd, g = random.Random(4), torch.Generator().manual_seed(4)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    lens, width = [0, 0, 0], 6
    free = list(range(40))
    rnd.shuffle(free)
    table = [[-1] * width for _ in lens]
    for step, adds in enumerate(([7, 5, 3], [1, 1, 1], [4, 0, 9], [1, 8, 1], [2, 2, 2])):
        total, B = sum(adds), sum(adds) + (1 if step % 2 else 0)  # some steps are padded
        bits = [b for a in adds for b in ref.tree_bits(rnd, a)] + [0] * (B - total)
        mask = ref.as_int64(bits)
        x = torch.randn(B, s.d, generator=g)
        dev_table = i32(table)
        want = ref.tables(lens, adds, table, free, page, B)
        got_x = x.to(DEV)
        t = spffn.block_tables(i32(lens), i32(adds), dev_table, i32(free), i32([len(free)]), page, B)
        assert t["slots"].tolist() == want["slots"] and dev_table.tolist() == want["table"]
        for l in range(layers):
            # each layer from the GPU's own input, so that a mask of the FFN's predictor that
            # falls the other way next to its border does not spread
            h_in = got_x.cpu().double()
            got = spffn.attn_step(s.attn[l], s.cache[l][0], got_x, t["starts"], i32(lens),
                                  t["slots"], dev_table, mask=mask.to(DEV), max_new=max(adds))
            c = s.cache[l][0]
            rows = ref.rows_of_k(c.k.cpu()), ref.rows_of_v(c.v.cpu())
            ref_h = host_layer(s, l, h_in, rows, want["starts"], lens, want["slots"],
                               dev_table.cpu(), mask, max(adds))
            # fp32 sums of 2 d + 16 and of 512 + 16 terms, each within a half step (2^-24) of
            # their magnitudes' sum, some sqrt(n) times the result: 6e-5 sqrt(512) = 1.4e-3
            err = (got.cpu().double() - ref_h)[:total]
            assert torch.equal(got[total:], got_x[total:])  # no request, no bias: x itself
            rel = err.norm() / (ref_h - h_in)[:total].norm()
            assert rel < 1.4e-3, (step, l, float(rel))
            h_mid = got.cpu().double().numpy()
            um = torch.empty(TINY.d_ffn, dtype=torch.uint8, device=DEV)
            got_x = spffn.decode_step(s.ffn[l], got, trace=dict(union_mask=um))
            o = oracle.decode_layer(s.np_ffn[l], h_mid, EPS, mask=um.cpu().numpy())
            y = got_x.cpu().double().numpy() - h_mid
            assert np.linalg.norm(y - o["y"]) <= 1e-3 * np.linalg.norm(o["y"])
        table, lens = want["table"], want["new_lens"]
        free = free[:want["left"][0]]


def test_graph_of_a_whole_step():
    s = Stack(2, torch.float16, seed=12)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    B, g = 6, torch.Generator().manual_seed(5)
    lens, adds = i32([20, 3]), i32([4, 1])
    table = i32([[1, 2, -1], [3, -1, -1]])
    free, n_free = i32([7, 8, 9]), i32([3])
    mask = ref.as_int64([1, 3, 5, 13, 1, 0]).to(DEV)
    x = torch.randn(B, s.d, generator=g).to(DEV)
    want, _ = s.step(x, lens, adds, table, free, n_free, B, mask, 4)  # warms up, fills the cache
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, t = s.step(x, lens, adds, table, free, n_free, B, mask, 4)
    for i, (ls, ads) in enumerate((([20, 3], [4, 1]), ([17, 30], [1, 4]), ([0, 16], [2, 3]))):
        x.copy_(torch.randn(B, s.d, generator=g))
        lens.copy_(i32(ls))
        adds.copy_(i32(ads))
        table.copy_(i32([[1, 2, -1], [3, 4, -1]]))
        caches = [(c.k.clone(), c.v.clone()) for c, _ in s.cache]
        want, tw = s.step(x, lens, adds, table, free, n_free, B, mask, 4)
        want = want.clone()
        for (c, _), (k, v) in zip(s.cache, caches):
            c.k.copy_(k)
            c.v.copy_(v)
        table.copy_(i32([[1, 2, -1], [3, 4, -1]]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(t["slots"], tw["slots"])


def test_in_place_and_out_of_place_agree():
    s = Stack(1, torch.float16, seed=13)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    x = torch.randn(3, s.d, device=DEV)
    args = (i32([0, 3]), i32([0]), i32([16, 17, 18]), i32([[1]]))
    a = spffn.attn_step(s.attn[0], s.cache[0][0], x, *args)
    h = x.clone()
    b = spffn.attn_step(s.attn[0], s.cache[0][0], h, *args, h=h)
    assert b is h and torch.equal(a, b)


def test_tokens_of_no_request_get_the_bias_alone():
    s = Stack(1, torch.float16, seed=14)
    at = s.attn[0]
    bias = torch.randn(s.d, device=DEV)
    s.cache[0][0].v.fill_(1.0)
    at = spffn.Attention(at.qkv, at.out, 8, 64, at.qkv_bias, bias)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    for B, R in ((5, 70), (16, 1), (7, 2000)):  # one request with a token, one with too many
        x = torch.randn(B, s.d, device=DEV)
        starts = torch.full((R + 1,), 4, dtype=torch.int32, device=DEV)
        starts[0] = 1
        ws = at.workspace(s.cache[0][0], B, 2).fill_(255)  # NaN wherever nothing is written
        h = spffn.attn_step(at, s.cache[0][0], x, starts, i32([3] * R), i32([-1] * B),
                            i32([[1]] * R), max_new=2, ws=ws)
        assert torch.isfinite(h).all()
        rest = [0] + list(range(3, B))
        # 0 W + bias + x, in either order of one fp32 addition
        assert torch.equal(h[rest], (x + bias)[rest])
        assert not torch.equal(h[1], (x + bias)[1])


def test_two_streams_at_once():
    # calls that overlap take a workspace each; what they compute is what they do alone
    stacks = [Stack(1, torch.float16, seed=15 + i) for i in range(2)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    x = torch.randn(6, stacks[0].d, device=DEV)
    args = (i32([0, 6]), i32([10]), i32(range(26, 32)), i32([[1]]))
    want = [spffn.attn_step(s.attn[0], s.cache[0][0], x, *args).clone() for s in stacks]
    streams, got = [torch.cuda.Stream() for _ in stacks], [None, None]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (s, stream) in enumerate(zip(stacks, streams)):
            with torch.cuda.stream(stream):
                got[i] = spffn.attn_step(s.attn[0], s.cache[0][0], x, *args)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_graphs_share_a_workspace():
    s = Stack(1, torch.float8_e4m3fn, seed=17)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    ws = s.attn[0].workspace(s.cache[0][0], 16, 8)
    runs = []
    for B in (5, 16):  # the two shapes of the product
        x = torch.randn(B, s.d, device=DEV)
        h = torch.empty_like(x)
        args = (i32([0, min(B, 8)]), i32([20]), i32([-1] * B), i32([[2, 5]]))
        call = lambda x=x, h=h, args=args: spffn.attn_step(  # noqa: E731
            s.attn[0], s.cache[0][0], x, *args, max_new=8, h=h, ws=ws)
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((x, h, call, graph))
    for i in range(3):
        for x, h, call, graph in runs:
            x.copy_(torch.randn(x.shape))
            want = call().clone()
            h.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, want), (i, x.shape[0])
