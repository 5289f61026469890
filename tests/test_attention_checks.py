"""The attention half's entry points refuse bad calls before anything is
enqueued: statuses of the C ABI on addresses that are never used, and the
binding's own checks on host tensors (size before device)."""
import ctypes as C

import pytest
import torch

import activation_sparse_mlp_amd as spffn
from activation_sparse_mlp_amd._lib import CacheDesc, Q4Desc

OK, E_ARG, E_SHAPE, E_DTYPE, E_WORKSPACE = 0, -1, -2, -3, -4
A = 0x10000000  # addresses far apart, never dereferenced


def at(i):
    return A + i * 0x10000000


def q4(**kw):
    d = dict(packed=at(0), rows=64, cols=256, group=64, zeros=0)
    d.update(kw)
    return Q4Desc(**d)


def matvec(w=None, **kw):
    a = dict(x=at(1), B=2, eps=-1.0, bias=None, resid=None, y=at(2), ws=at(4), nb=1 << 20)
    a.update(kw)
    w = q4() if w is None else w
    return spffn.load().spffn_q4_matvec(C.byref(w), a["x"], a["B"], a["eps"], a["bias"],
                                        a["resid"], a["y"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("status,call", [
    (E_ARG, lambda: matvec(q4(packed=None))),
    (E_ARG, lambda: matvec(q4(packed=at(0) + 8))),
    (E_SHAPE, lambda: matvec(q4(rows=0))),
    (E_SHAPE, lambda: matvec(q4(rows=(1 << 24) + 1))),
    (E_SHAPE, lambda: matvec(q4(cols=48))),
    (E_SHAPE, lambda: matvec(q4(cols=0))),
    (E_SHAPE, lambda: matvec(q4(cols=(1 << 20) + 32))),
    (E_SHAPE, lambda: matvec(q4(group=16))),
    (E_SHAPE, lambda: matvec(B=0)),
    (E_SHAPE, lambda: matvec(B=17)),
    (E_ARG, lambda: matvec(x=None)),
    (E_ARG, lambda: matvec(x=at(1) + 4)),
    (E_ARG, lambda: matvec(y=None)),
    (E_ARG, lambda: matvec(y=at(1) + 64)),                 # y inside x
    (E_ARG, lambda: matvec(resid=at(2) + 16)),             # part of y
    (E_ARG, lambda: matvec(bias=at(2) + 128)),
    (E_ARG, lambda: matvec(bias=at(3) + 2)),
    (E_ARG, lambda: matvec(eps=float("nan"))),
    (E_ARG, lambda: matvec(eps=float("inf"))),
    (E_WORKSPACE, lambda: matvec(B=3, ws=None)),
    (E_WORKSPACE, lambda: matvec(B=3, nb=4096)),
    (E_ARG, lambda: matvec(B=9, ws=at(4) + 64)),
])
def test_matvec(status, call):
    assert call() == status
    assert spffn.load().spffn_last_error()


def test_pack():
    lib = spffn.load()
    pack = lib.spffn_q4_pack
    assert pack(None, at(1), None, 4, 64, 32, at(2), None) == E_ARG
    assert pack(at(0), None, None, 4, 64, 32, at(2), None) == E_ARG
    assert pack(at(0), at(1), None, 4, 64, 32, None, None) == E_ARG
    assert pack(at(0), at(1), None, 4, 64, 32, at(2) + 4, None) == E_ARG
    assert pack(at(0), at(1), None, 4, 63, 32, at(2), None) == E_SHAPE
    assert pack(at(0), at(1), None, -4, 64, 32, at(2), None) == E_SHAPE
    assert pack(at(0), at(1), None, 4, 64, 48, at(2), None) == E_SHAPE
    assert pack(at(0), at(1), None, 4, 64, 32, at(0), None) == E_ARG       # in place
    assert pack(at(0), at(1), at(2) + 16, 4, 64, 32, at(2), None) == E_ARG
    # rows and columns are padded to 16 and 128
    nb = lib.spffn_q4_packed_bytes
    assert nb(1, 32, 128, 0) == 1024 + 32 and nb(17, 160, 32, 1) == 4 * (1024 + 4 * 48)
    assert nb(0, 32, 32, 0) == nb(1, 40, 32, 0) == nb(1, 32, 8, 0) == 0


def test_matvec_workspace_bytes():
    nb = spffn.load().spffn_q4_matvec_workspace_bytes
    w = C.byref(q4())
    assert nb(w, 1) == nb(w, 2) == nb(w, 0) == nb(w, 17) == nb(None, 3) == 0
    assert 0 < nb(w, 3) <= nb(w, 8) < nb(w, 9) <= nb(w, 16)
    assert nb(C.byref(q4(cols=40)), 4) == 0


def tables(**kw):
    a = dict(lens=at(0), adds=at(1), R=4, page=16, table=at(2), width=8, free=at(3), cap=10,
             n_free=at(4), starts=at(5), new_lens=at(6), slots=at(7), positions=at(8), N=9,
             left=at(9))
    a.update(kw)
    return spffn.load().spffn_block_tables(
        a["lens"], a["adds"], a["R"], a["page"], a["table"], a["width"], a["free"], a["cap"],
        a["n_free"], a["starts"], a["new_lens"], a["slots"], a["positions"], a["N"], a["left"],
        None)


@pytest.mark.parametrize("status,kw", [
    *[(E_ARG, {k: None}) for k in ("lens", "adds", "table", "free", "n_free", "starts", "new_lens",
                                   "slots", "positions", "left")],
    (E_ARG, dict(lens=at(0) + 2)), (E_ARG, dict(left=at(9) + 1)),
    (E_SHAPE, dict(R=0)), (E_SHAPE, dict(R=4097)), (E_SHAPE, dict(page=8)),
    (E_SHAPE, dict(page=48)), (E_SHAPE, dict(page=512)), (E_SHAPE, dict(width=0)),
    (E_SHAPE, dict(cap=-1)), (E_SHAPE, dict(N=-1)),
    (E_ARG, dict(new_lens=at(0))),              # lengths in place
    (E_ARG, dict(left=at(4))),                  # the free count in place
    (E_ARG, dict(slots=at(8) + 32)),            # two outputs
    (E_ARG, dict(table=at(3) + 36)),
])
def test_block_tables(status, kw):
    assert tables(**kw) == status
    assert spffn.load().spffn_last_error()


def cache(**kw):
    d = dict(k=at(0), v=at(1), k_scale=None, v_scale=None, pages=10, page_size=16, kv_heads=2,
             head_dim=64, dtype=1)
    d.update(kw)
    return CacheDesc(**d)


BAD_CACHES = [
    (E_ARG, dict(k=None)), (E_ARG, dict(v=at(1) + 8)), (E_DTYPE, dict(dtype=0)),
    (E_DTYPE, dict(dtype=2)), (E_ARG, dict(dtype=3)), (E_ARG, dict(k_scale=at(2))),
    (E_ARG, dict(dtype=3, k_scale=at(2))), (E_ARG, dict(dtype=3, k_scale=at(2), v_scale=at(3) + 2)),
    (E_SHAPE, dict(page_size=8)), (E_SHAPE, dict(page_size=24)), (E_SHAPE, dict(page_size=512)),
    (E_SHAPE, dict(head_dim=80)), (E_SHAPE, dict(kv_heads=0)), (E_SHAPE, dict(pages=0)),
    (E_SHAPE, dict(pages=1 << 27)),
]


def append(c, **kw):
    a = dict(k=at(4), v=at(5), dtype=0, ld_k=128, ld_v=128, slots=at(6), N=3)
    a.update(kw)
    return spffn.load().spffn_kv_append(C.byref(c), a["k"], a["v"], a["dtype"], a["ld_k"],
                                        a["ld_v"], a["slots"], a["N"], None)


def attend(c, **kw):
    a = dict(q=at(4), dtype=0, ld_q=256, N=5, heads=4, starts=at(5), lens=at(6), table=at(7), R=2,
             width=9, mask=at(8), max_new=4, scale=0.1, out=at(9), ld_out=256, ws=at(10),
             nb=1 << 27)
    a.update(kw)
    return spffn.load().spffn_tree_attention(
        C.byref(c), a["q"], a["dtype"], a["ld_q"], a["N"], a["heads"], a["starts"], a["lens"],
        a["table"], a["R"], a["width"], a["mask"], a["max_new"], a["scale"], a["out"], a["ld_out"],
        a["ws"], a["nb"], None)


@pytest.mark.parametrize("status,kw", BAD_CACHES)
def test_cache(status, kw):
    assert append(cache(**kw)) == status
    assert attend(cache(**kw)) == status
    assert spffn.load().spffn_tree_attention_workspace_bytes(C.byref(cache(**kw)), 4, 4, 0) == 0
    assert spffn.load().spffn_kv_append(None, at(4), at(5), 0, 128, 128, at(6), 3, None) == E_ARG


@pytest.mark.parametrize("status,kw", [
    (E_ARG, dict(k=None)), (E_ARG, dict(v=None)), (E_ARG, dict(slots=None)),
    (E_ARG, dict(k=at(4) + 8)), (E_ARG, dict(slots=at(6) + 2)), (E_DTYPE, dict(dtype=3)),
    (E_SHAPE, dict(ld_k=124)), (E_ARG, dict(ld_v=130)), (E_ARG, dict(dtype=1, ld_v=132)),
    (E_SHAPE, dict(N=-1)), (OK, dict(N=0, k=None)),
])
def test_append(status, kw):
    assert append(cache(), **kw) == status


@pytest.mark.parametrize("status,kw", [
    *[(E_ARG, {k: None}) for k in ("q", "out", "starts", "lens", "table")],
    (E_ARG, dict(q=at(4) + 8)), (E_ARG, dict(mask=at(8) + 4)), (E_ARG, dict(ld_q=258)),
    (E_SHAPE, dict(ld_out=128)), (E_DTYPE, dict(dtype=2)), (E_SHAPE, dict(heads=3)),
    (E_SHAPE, dict(heads=0)), (E_SHAPE, dict(max_new=0)), (E_SHAPE, dict(max_new=65)),
    (E_SHAPE, dict(R=0)), (E_SHAPE, dict(R=4097)), (E_SHAPE, dict(width=0)),
    (E_SHAPE, dict(width=1 << 30)), (E_SHAPE, dict(N=-1)), (E_ARG, dict(scale=float("nan"))),
    (E_ARG, dict(scale=float("inf"))), (E_ARG, dict(out=at(4))),
    (E_ARG, dict(out=at(4) + 4 * 1024)),                     # the last row of q
    (E_WORKSPACE, dict(ws=None)), (E_WORKSPACE, dict(nb=1024)), (E_ARG, dict(ws=at(10) + 16)),
    (OK, dict(N=0, q=None, out=None)),
])
def test_attention(status, kw):
    assert attend(cache(), **kw) == status


def test_workspace_bytes():
    nb = spffn.load().spffn_tree_attention_workspace_bytes
    ref = C.byref(cache())
    assert 0 < nb(ref, 4, 1, 0) <= nb(ref, 4, 64, 0)
    for heads, new, dtype in ((3, 1, 0), (0, 1, 0), (4, 0, 0), (4, 65, 0), (4, 1, 3)):
        assert nb(ref, heads, new, dtype) == 0


def attn_step(**kw):
    from activation_sparse_mlp_amd._lib import AttnDesc
    a = dict(rows=(4 + 2 * 2) * 64, cols=96, out_rows=96, out_cols=256, heads=4, eps=1e-5, scale=0.1,
             qkv_packed=at(2), out_packed=at(3), qkv_bias=None, x=at(4), h=at(5), B=3, slots=at(6),
             starts=at(7), lens=at(8), table=at(9), R=2, width=5, mask=None, max_new=3, ws=at(10),
             nb=1 << 27)
    a.update(kw)
    d = AttnDesc(qkv=q4(packed=a["qkv_packed"], rows=a["rows"], cols=a["cols"]),
                 out=q4(packed=a["out_packed"], rows=a["out_rows"], cols=a["out_cols"]),
                 qkv_bias=a["qkv_bias"], heads=a["heads"], rms_eps=a["eps"], scale=a["scale"])
    return spffn.load().spffn_attn_step(
        C.byref(d), C.byref(cache()), a["x"], a["h"], a["B"], a["slots"], a["starts"], a["lens"],
        a["table"], a["R"], a["width"], a["mask"], a["max_new"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("status,kw", [
    *[(E_ARG, {k: None}) for k in ("x", "h", "slots", "starts", "lens", "table", "qkv_packed",
                                   "out_packed")],
    (E_ARG, dict(h=at(4) + 64)), (E_ARG, dict(x=at(4) + 4)), (E_ARG, dict(eps=-1.0)),
    (E_ARG, dict(scale=float("nan"))), (E_ARG, dict(qkv_bias=at(1) + 2)),
    (E_SHAPE, dict(B=0)), (E_SHAPE, dict(B=17)), (E_SHAPE, dict(heads=3)),
    (E_SHAPE, dict(rows=512 + 16)), (E_SHAPE, dict(out_cols=288)), (E_SHAPE, dict(out_rows=128)),
    (E_SHAPE, dict(max_new=65)), (E_SHAPE, dict(R=0)), (E_SHAPE, dict(width=0)),
    (E_WORKSPACE, dict(ws=None)), (E_WORKSPACE, dict(nb=4096)),
])
def test_attn_step(status, kw):
    assert attn_step(**kw) == status
    assert spffn.load().spffn_last_error()


# --------------------------------------------------------------------------- binding
def _u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


@pytest.mark.parametrize("args,kw", [
    ((_u8(4, 24), torch.zeros(4, 2).half()), {}),                    # 48 columns
    ((_u8(4, 32), torch.zeros(4, 3).half()), {}),                    # 64 / 32 groups are 2
    ((_u8(4, 32), torch.zeros(4, 2).half(), _u8(4, 1)), {}),
    ((_u8(4, 32), torch.zeros(4, 2).half()), dict(group=16)),
    ((_u8(0, 32), torch.zeros(0, 2).half()), {}),
    ((_u8(128), torch.zeros(4, 2).half()), {}),
])
def test_q4_matrix_sizes(args, kw):
    with pytest.raises(ValueError):
        spffn.Q4Matrix(*args, **kw)


def test_q4_matrix_needs_a_device():
    with pytest.raises(TypeError, match="CUDA"):
        spffn.Q4Matrix(_u8(4, 32), torch.zeros(4, 2).half())


class FakeMatrix:
    rows, cols, device, _index, _need = 8, 64, torch.device("cuda:0"), 0, [0] * 17


@pytest.mark.parametrize("x,kw", [
    (torch.zeros(2, 65), {}), (torch.zeros(2, 2, 64), {}), (torch.zeros(17, 64), {}),
    (torch.zeros(0, 64), {}),
    (torch.zeros(2, 64), dict(bias=torch.zeros(9))),
    (torch.zeros(2, 64), dict(resid=torch.zeros(8))),
    (torch.zeros(2, 64), dict(y=torch.zeros(2, 9))),
    (torch.zeros(2, 64), dict(rms_eps=-1.0)),
    (torch.zeros(2, 64), dict(rms_eps=float("nan"))),
])
def test_q4_matvec_sizes(x, kw):
    with pytest.raises(ValueError):
        spffn.q4_matvec(FakeMatrix, x, **kw)


@pytest.mark.parametrize("kw", [
    dict(adds=_i(2)), dict(table=_i(2, 4)), dict(table=_i(12)), dict(n_free=_i(2)),
    dict(starts=_i(3)), dict(new_lens=_i(4)), dict(slots=_i(6)), dict(positions=_i(4)),
    dict(left=_i(1)), dict(n_tokens=-1),
])
def test_block_tables_sizes(kw):
    a = dict(lens=_i(3), adds=_i(3), table=_i(3, 4), free_list=_i(5), n_free=_i(1), page_size=16,
             n_tokens=5)
    a.update(kw)
    with pytest.raises(ValueError):
        spffn.block_tables(**a)


def _k(pages=2, H=2, n=8, page=16, E=8, dtype=torch.float16):
    return torch.zeros(pages, H, n, page, E).to(dtype)


@pytest.mark.parametrize("args", [
    (_k(E=4), _k()), (_k(n=10), torch.zeros(2, 2, 2, 80, 8).half()), (_k(page=24), _k()),
    (_k(), _k()), (_k(), torch.zeros(2, 2, 2, 64, 8).half(), torch.ones(2), torch.ones(2)),
    (_k(n=4, E=16, dtype=torch.float8_e4m3fn), torch.zeros(2, 2, 1, 64, 16)),
])
def test_kv_cache_shapes(args):
    with pytest.raises(ValueError):
        spffn.KVCache(*args)


def test_kv_cache_dtype():
    with pytest.raises(TypeError):
        spffn.KVCache(torch.zeros(2, 2, 8, 16, 8), torch.zeros(2, 2, 2, 64, 8))


class FakeCache:
    kv_heads, head_dim, device, _index = 2, 64, torch.device("cuda:0"), 0


def test_rows_and_counts():
    q = torch.zeros(4, 4, 64)
    ok = dict(starts=_i(3), lens=_i(2), table=_i(2, 5))
    for bad in (dict(q=torch.zeros(4, 3, 64)), dict(q=torch.zeros(4, 4, 32)),
                dict(q=torch.zeros(4, 256)), dict(starts=_i(2)), dict(table=_i(3, 5)),
                dict(mask=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            spffn.tree_attention(FakeCache, **{**dict(q=q), **ok, **bad})
    with pytest.raises((ValueError, TypeError)):
        spffn.kv_append(FakeCache, torch.zeros(3, 2, 32), torch.zeros(3, 2, 64), _i(3))
    with pytest.raises(TypeError, match="CUDA"):
        spffn.kv_append(FakeCache, torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), _i(3))


# --------------------------------------------------------------------------- memory that overlaps
@pytest.mark.parametrize("call", [
    lambda c: append(c, k=c.k + 256), lambda c: append(c, v=c.v), lambda c: append(c, k=c.v),
    lambda c: append(c, k=c.k - 128 * 4 * 2),              # the last row of three
    lambda c: append(c, slots=c.k + 16),
    lambda c: attend(c, out=c.v + 512), lambda c: attend(c, out=c.k),
    lambda c: attend(c, ws=at(9)), lambda c: attend(c, ws=at(4)), lambda c: attend(c, ws=c.k),
    lambda c: matvec(B=5, ws=at(1)), lambda c: matvec(B=5, ws=at(2)),
    lambda c: attn_step(ws=at(4)), lambda c: attn_step(ws=at(5)), lambda c: attn_step(ws=c.v),
    lambda c: attn_step(x=c.k, h=c.k),
])
def test_overlaps(call):
    assert call(cache()) == E_ARG
    assert "overlap" in spffn.load().spffn_last_error().decode()
