"""Block tables, slot maps and the append to a paged cache against plain host
forms: shortages, requests that do not fit, empty ones, padding, runs of slots
that start and end anywhere, strided rows, both cache types, saturation."""
import random

import pytest
import torch

import activation_sparse_mlp_amd as spffn
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def run_tables(lens, adds, table, free, page, n, cap_extra=0):
    t = i32(table)
    got = spffn.block_tables(i32(lens), i32(adds), t, i32(free + [12345] * cap_extra),
                             i32([len(free)]), page, n)
    torch.cuda.synchronize()
    return {**{k: v.tolist() for k, v in got.items()}, "table": t.tolist()}


def problem(rnd, R, page, most_len, most_add, free_share):
    lens = [rnd.choice([0, 1, page - 1, page, rnd.randint(0, most_len)]) for _ in range(R)]
    lens = [min(v, most_len) for v in lens]
    adds = [rnd.choice([0, 1, rnd.randint(0, most_add)]) for _ in range(R)]
    width = -(-(most_len + most_add) // page)
    ids = list(range(R * width + 50))
    rnd.shuffle(ids)
    table = []
    for t in lens:
        row = [-1] * width
        for b in range(-(-t // page)):
            row[b] = ids.pop()
        table.append(row)
    need = sum(-(-(t + a) // page) - -(-t // page) for t, a in zip(lens, adds))
    free = ids[:int(need * free_share) + (3 if free_share >= 1 else 0)]
    return lens, adds, table, free


@pytest.mark.parametrize("R,page,most_len,most_add,share", [
    (1, 16, 40, 3, 1.0), (1, 16, 0, 1, 1.0), (2, 256, 700, 300, 1.0), (16, 16, 300, 1, 1.0),
    (63, 32, 200, 40, 1.0), (256, 16, 100, 20, 0.5), (257, 64, 500, 70, 0.0),
    (700, 128, 900, 257, 0.9), (4096, 16, 64, 5, 0.97),
])
def test_tables(R, page, most_len, most_add, share):
    rnd = random.Random(R * 7 + page)
    lens, adds, table, free = problem(rnd, R, page, most_len, most_add, share)
    for pad in (0, 5):
        n = sum(adds) + pad
        want = ref.tables(lens, adds, table, free, page, n)
        got = run_tables(lens, adds, table, free, page, n, cap_extra=pad)
        for k in want:
            assert got[k] == want[k], k


def test_tables_requests_that_cannot_be_written():
    page, width = 16, 2
    lens = [-3, 5, 20, 30, 0, 32, 31, 2]
    adds = [2, -1, 13, 2, 0, 0, 1, 15]
    table = [[-1, -1], [3, -1], [4, 5], [6, 7], [-1, -1], [8, 9], [10, 11], [12, -1]]
    free = [20, 21]
    want = ref.tables(lens, adds, table, free, page, 40)
    got = run_tables(lens, adds, table, free, page, 40)
    for k in want:
        assert got[k] == want[k], k
    assert got["left"] == [1, 3] and got["table"][7] == [12, 21]


def test_tables_unmapped_entry_gives_no_slot():
    got = run_tables([17, 3], [2, 1], [[4, -1], [-1, 7]], [9], 16, 3)
    assert got["slots"] == [-1, -1, -1]  # pages that the tables should hold and do not
    assert got["left"] == [1, 0]


def test_tables_shorter_slot_buffer_and_no_tokens():
    lens, adds, table = [0, 16], [20, 4], [[-1, -1], [5, -1]]
    want = ref.tables(lens, adds, table, [1, 2, 3], 16, 7)
    got = run_tables(lens, adds, table, [1, 2, 3], 16, 7)
    for k in want:
        assert got[k] == want[k], k
    got = run_tables(lens, [0, 0], table, [], 16, 0)
    assert got["starts"] == [0, 0, 0] and got["left"] == [0, 0] and got["slots"] == []


def test_tables_graph_replays():
    page, R, n = 16, 5, 12
    lens, adds = i32([0, 15, 16, 40, 3]), i32([1, 2, 0, 3, 4])
    first = [[-1] * 4, [1, -1, -1, -1], [2, -1, -1, -1], [3, 4, 5, -1], [6, -1, -1, -1]]
    table, free, n_free = i32(first), i32([10, 11, 12, 13]), i32([4])
    out = spffn.block_tables(lens, adds, table, free, n_free, page, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spffn.block_tables(lens, adds, table, free, n_free, page, n, **out)
    rnd = random.Random(1)
    for _ in range(4):
        ls, ads = [rnd.randint(0, 40) for _ in range(R)], [rnd.randint(0, 2) for _ in range(R)]
        rows = [[7 * r + b if b < -(-t // page) else -1 for b in range(4)] for r, t in
                enumerate(ls)]
        lens.copy_(i32(ls))
        adds.copy_(i32(ads))
        table.copy_(i32(rows))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.tables(ls, ads, rows, [10, 11, 12, 13], page, n)
        for k in out:
            assert out[k].tolist() == want[k], k
        assert table.tolist() == want["table"]


# --------------------------------------------------------------------------- append
CACHE = [torch.float16, torch.float8_e4m3fn]


def empty_cache(dtype, pages, H, D, page, seed):
    g = torch.Generator().manual_seed(seed)
    E = ref.packet(dtype)
    k = torch.randn(pages, H, D // E, page, E, generator=g).to(dtype)
    v = torch.randn(pages, H, page // E, D, E, generator=g).to(dtype)
    scales = (None, None)
    if E == 16:
        scales = (torch.rand(H, generator=g) * 0.1 + 0.01, torch.rand(H, generator=g) + 0.1)
    cache = spffn.KVCache(k.to(DEV), v.to(DEV), *(None if s is None else s.to(DEV)
                                                  for s in scales))
    return cache, k, v, scales, g


def check_append(dtype, src, H, D, page, pages, slots, strided, seed, big=False):
    cache, k, v, (ks, vs), g = empty_cache(dtype, pages, H, D, page, seed)
    N = len(slots)
    buf = torch.randn(N, 2 * H + (3 if strided else 0), D, generator=g)
    if big:
        buf[0, :, 0] = float("nan")
        buf[0, :, 1] = float("inf")
        buf[N // 2, :, 2] = -1e6
        buf[N - 1, :, 3] = 1e-9
    buf = buf.to(src).to(DEV)
    nk, nv = buf[:, 1:1 + H] if strided else buf[:, :H], buf[:, -H:]
    if not strided:
        nk, nv = nk.contiguous(), nv.contiguous()
    spffn.kv_append(cache, nk, nv, i32(slots))
    torch.cuda.synchronize()
    kr, vr = ref.rows_of_k(k).clone(), ref.rows_of_v(v).clone()
    raw = torch.uint8 if dtype != torch.float16 else torch.int16
    for rows, new, scale in ((kr, nk, ks), (vr, nv, vs)):
        got = ref.round_rows(new.cpu(), dtype, scale).view(raw)
        for n, s in enumerate(slots):
            if 0 <= s < pages * page:
                rows.view(raw)[s] = got[n]
    # bit for bit, written rows and the others (NaN by its place: its bits may differ)
    for got, rows in ((ref.rows_of_k(cache.k.cpu()), kr), (ref.rows_of_v(cache.v.cpu()), vr)):
        nan = rows.float().isnan()
        assert torch.equal(got.float().isnan(), nan)
        assert torch.equal(got.view(raw)[~nan], rows.view(raw)[~nan])


@pytest.mark.parametrize("dtype", CACHE)
@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("H,D,page", [(1, 64, 16), (2, 96, 32), (3, 128, 64), (8, 256, 128)])
def test_append_scattered_and_runs(dtype, src, H, D, page):
    rnd = random.Random(D + page)
    pages = 6
    every = list(range(pages * page))
    scattered = rnd.sample(every, 21)
    check_append(dtype, src, H, D, page, pages, scattered, True, 1)
    run = list(range(5, 5 + 37))                    # starts and ends inside packets
    check_append(dtype, src, H, D, page, pages, run, True, 2)
    aligned = list(range(2 * page, 2 * page + 16)) + list(range(16))
    check_append(dtype, src, H, D, page, pages, aligned, False, 3)
    holes = [3, 4, -1, 6, 7, 8, pages * page, 9, 10, -5, 2 ** 31 - 1, 15, 14, 13, 31, 30]
    check_append(dtype, src, H, D, page, pages, holes, True, 4)
    check_append(dtype, src, H, D, page, pages, [7], True, 5)


@pytest.mark.parametrize("dtype", CACHE)
def test_append_extremes(dtype):
    check_append(dtype, torch.float32, 2, 64, 16, 4, list(range(40)), True, 6, big=True)


def test_append_quotients_at_the_borders():
    # every E4M3 border (the value half way between two neighbours) and its fp32 neighbours,
    # times scales of all sizes: the quotient decides the code, so it has to be exact
    codes = torch.arange(0, 0x7E, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    nxt = torch.arange(1, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    g = torch.Generator().manual_seed(9)
    H, D, page = 8, 64, 16
    scales = torch.tensor([1.0, 0.1, 3.7e-5, 7.0, 1e-20, 3e19, 0.3333333, 1.7e6])
    rows = []
    for h in range(H):
        x = (codes + nxt) / 2 * scales[h]
        ulp = x.abs() * 2.0 ** -23
        x = torch.cat([x, x + ulp, x - ulp, -x, x + 2 * ulp, x - 2 * ulp,
                       torch.randn(5 * 126, generator=g) * scales[h] * 100])
        rows.append(x[:21 * D].view(21, D) if x.numel() >= 21 * D else
                    torch.cat([x, x.new_zeros(21 * D - x.numel())]).view(21, D))
    new = torch.stack(rows, 1).contiguous()
    k = torch.zeros(2, H, D // 16, page, 16).to(torch.float8_e4m3fn).to(DEV)
    v = torch.zeros(2, H, page // 16, D, 16).to(torch.float8_e4m3fn).to(DEV)
    cache = spffn.KVCache(k, v, scales.to(DEV), scales.to(DEV))
    spffn.kv_append(cache, new.to(DEV), new.to(DEV), i32(list(range(21))))
    torch.cuda.synchronize()
    want = ref.round_rows(new, torch.float8_e4m3fn, scales).view(torch.uint8)
    assert torch.equal(ref.rows_of_k(k.cpu())[:21].view(torch.uint8), want)
    assert torch.equal(ref.rows_of_v(v.cpu())[:21].view(torch.uint8), want)


@pytest.mark.parametrize("dtype", CACHE)
@pytest.mark.parametrize("src", [torch.float32, torch.float16])
@pytest.mark.parametrize("H,D,start", [(2, 128, 7), (9, 128, 7), (8, 64, 16), (8, 96, 0), (9, 256, 9)])
def test_append_prompt(dtype, src, H, D, start):
    # 2001 tokens of two heads go in small workgroups, those of eight in large ones
    page, pages = 32, 70
    order = list(range(pages))
    random.Random(3).shuffle(order)
    at = lambda i: order[(i + start) // page] * page + (i + start) % page  # noqa: E731
    slots = [at(i) for i in range(2101)]
    slots[100] = -1
    slots[640:660] = [at(i) for i in range(659, 639, -1)]  # backwards: no packet is whole
    slots[1203], slots[1209] = slots[1209], slots[1203]
    check_append(dtype, src, H, D, page, pages, slots, True, 7)


def test_append_far_offsets():
    # a cache past 2^31 elements: rows near its end are where they should be
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (H * D * page) + 3
    E = 16
    k = torch.zeros(pages, H, D // E, page, E, dtype=torch.float8_e4m3fn, device=DEV)
    v = torch.zeros(pages, H, page // E, D, E, dtype=torch.float8_e4m3fn, device=DEV)
    one = torch.ones(H, device=DEV)
    cache = spffn.KVCache(k, v, one, one)
    new = torch.ones(2, H, D, device=DEV)
    spffn.kv_append(cache, new, 2 * new, i32([pages * page - 1, 0]))
    torch.cuda.synchronize()
    assert bool((k[-1, :, :, -1].float() == 1).all()) and bool((v[-1, :, -1, :, -1].float() == 2).all())
    assert bool((k[0, :, :, 0].float() == 1).all()) and bool((v[0, :, 0, :, 0].float() == 2).all())
    assert int(k.view(torch.int64).count_nonzero()) == 2 * H * D // 8
    assert float(v[-1].float().sum()) == 2 * H * D
