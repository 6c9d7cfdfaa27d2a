"""The recurrent-block calls without a GPU: every refusal happens on the host, before any HIP call."""
import ctypes

import pytest
import torch

from sequence_state_scan_amd import gla

E, UN = gla.GLA_ERR_INVALID_ARG, gla.GLA_ERR_UNSUPPORTED


def p(i):
    return ctypes.c_void_p(0x10000 * (i + 1))  # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    return gla.load_library()


def strides(*v):
    return (ctypes.c_longlong * 3)(*v)


def call(fn, names, defaults, **kw):
    bad = set(kw) - set(names)
    assert not bad, bad
    return fn(*[kw[n] if n in kw else defaults[n] for n in names])


def _table(ptrs, ints, tail):
    names = ptrs + list(ints) + list(tail)
    d = {n: None if n.endswith("_st") else p(i) for i, n in enumerate(ptrs)}
    d.update(ints)
    d.update(tail)
    return names, d


RECUR_FWD = _table(["x", "x_st", "g", "g_st", "h0", "lens", "h", "chunk_in", "h_final"],
                   dict(B=2, T=300, D=64, mode=0, dtype=1), dict(ws=p(30), wsb=1 << 30, stream=None))
RECUR_BWD = _table(["x", "x_st", "g", "g_st", "dh", "dh_st", "chunk_in", "lens", "dhT", "dx", "dg", "dh0"],
                   dict(B=2, T=300, D=64, mode=0, dtype=1), dict(ws=p(30), wsb=1 << 30, stream=None))
RECUR_STEP = _table(["x", "x_st", "g", "g_st", "state", "slots", "h"], dict(B=2, D=64, n_slots=4, mode=0, dtype=1),
                    dict(stream=None))
STEP = _table(["q", "q_st", "k", "k_st", "v", "v_st", "g", "g_st", "state", "slots", "o"],
              dict(B=2, H=2, n=1, dk=64, dv=64, n_slots=4, dtype=1), dict(stream=None))
JOIN_FWD = _table(["y", "y_st", "z", "z_st", "w_post", "residual", "r_st", "scale", "w_pre", "out", "normed",
                   "rstd_post", "rstd_pre"], dict(B=2, H=2, T=10, d=64, act=0, eps=1e-6, dtype=1, stream_dtype=1),
                  dict(stream=None))
JOIN_BWD = _table(["y", "y_st", "z", "z_st", "w_post", "residual", "r_st", "scale", "w_pre", "rstd_post", "rstd_pre",
                   "d_out", "do_st", "d_normed", "dn_st", "dy", "dz", "d_residual", "dw_post", "dscale", "dw_pre"],
                  dict(B=2, H=2, T=10, d=64, act=0, dtype=1, stream_dtype=1),
                  dict(ws=p(30), wsb=1 << 30, stream=None))


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), E), (dict(T=0), E), (dict(D=0), E), (dict(mode=3), E), (dict(mode=-1), E), (dict(dtype=2), E),
    (dict(x=None), E), (dict(g=None), E), (dict(h=None), E), (dict(h=p(0)), E), (dict(chunk_in=p(6)), E),
    (dict(h_final=p(4)), E), (dict(x_st=strides(-1, 0, 64)), E), (dict(g_st=strides(0, 0, -64)), E), (dict(B=70000), UN),
    (dict(ws=p(0)), E), (dict(ws=None), E), (dict(wsb=16), E), (dict(ws=ctypes.c_void_p(0x300004)), E),
    (dict(D=1 << 24), UN), (dict(x_st=strides(1 << 30, 0, 1 << 24)), UN), (dict(B=60000, T=1 << 20), UN)])
def test_recur_fwd_refusals(lib, kw, want):
    assert call(lib.gla_recur_fwd, *RECUR_FWD, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_recur_fwd: ")


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), E), (dict(T=0), E), (dict(mode=9), E), (dict(dtype=5), E), (dict(dh=None), E), (dict(chunk_in=None), E),
    (dict(dx=None), E), (dict(dg=None), E), (dict(dx=p(4)), E), (dict(dg=p(9)), E), (dict(dh0=p(8)), E),
    (dict(dh_st=strides(0, 0, -1)), E), (dict(dh_st=strides(0, 0, 1 << 24)), UN), (dict(ws=None), E), (dict(wsb=16), E)])
def test_recur_bwd_refusals(lib, kw, want):
    assert call(lib.gla_recur_bwd, *RECUR_BWD, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_recur_bwd: ")


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), E), (dict(D=0), E), (dict(state=None), E), (dict(h=None), E), (dict(n_slots=0), E), (dict(mode=3), E),
    (dict(slots=None, n_slots=1), E), (dict(h=p(4)), E), (dict(state=p(0)), E), (dict(x_st=strides(-64, 0, 0)), E)])
def test_recur_step_refusals(lib, kw, want):
    assert call(lib.gla_recur_step, *RECUR_STEP, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_recur_step: ")


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), E), (dict(H=0), E), (dict(n=0), E), (dict(dk=0), E), (dict(dv=0), E), (dict(dtype=3), E),
    (dict(q=None), E), (dict(state=None), E), (dict(o=None), E), (dict(slots=None, n_slots=1), E), (dict(dk=257), UN),
    (dict(o=p(0)), E), (dict(state=p(4)), E), (dict(v_st=strides(0, 0, -1)), E),
    (dict(B=1 << 20, H=1 << 10, n_slots=1 << 21), UN)])
def test_step_refusals(lib, kw, want):
    assert call(lib.gla_step, *STEP, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_step: ")


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), E), (dict(d=0), E), (dict(act=2), E), (dict(eps=0.0), E), (dict(eps=-1.0), E), (dict(eps=float("nan")), E),
    (dict(dtype=4), E), (dict(stream_dtype=4), E), (dict(dtype=0, stream_dtype=1), UN), (dict(H=64, d=129), UN),
    (dict(y=None), E), (dict(out=None), E), (dict(normed=None), E), (dict(w_pre=None), E),
    (dict(w_post=None), E), (dict(out=p(0)), E), (dict(normed=p(5)), E), (dict(out=p(10)), E),
    (dict(out=p(5), r_st=strides(1280, 0, 256)), E), (dict(y_st=strides(0, -1, 0)), E)])
def test_join_fwd_refusals(lib, kw, want):
    assert call(lib.gla_join_fwd, *JOIN_FWD, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_join_fwd: ")


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), E), (dict(act=-1), E), (dict(dtype=0, stream_dtype=1), UN), (dict(H=1, d=8193), UN), (dict(y=None), E),
    (dict(dy=None), E), (dict(d_out=None, d_normed=None), E), (dict(w_pre=None, dw_pre=None), E), (dict(rstd_pre=None), E),
    (dict(rstd_post=None), E), (dict(w_post=None, dw_post=None), E), (dict(dz=None), E), (dict(z=None), E),
    (dict(scale=None), E), (dict(residual=None), E), (dict(ws=None), E), (dict(wsb=16), E), (dict(dy=p(11)), E),
    (dict(dz=p(15)), E), (dict(do_st=strides(-1, 0, 0)), E)])
def test_join_bwd_refusals(lib, kw, want):
    assert call(lib.gla_join_bwd, *JOIN_BWD, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_join_bwd: ")


def test_sizes(lib):
    assert lib.gla_recur_workspace_size(0, 5, 5) == 0 and lib.gla_last_error()
    gla.recur_workspace_size(1, 1, 1)
    with pytest.raises(gla.GLAError):
        gla.recur_workspace_size(1, 0, 1)
    assert lib.gla_join_workspace_size(1, 1, 1, 0) == 0
    assert gla.join_workspace_size(2, 4, 100, 64) >= 100 * 3 * 256 * 4 // 32
    with pytest.raises(gla.GLAError):
        gla.join_workspace_size(1, 2, 1, 5000)


@pytest.mark.parametrize("H,d", [(2049, 3), (4096, 2), (2049, 1), (8192, 1)])
def test_join_refuses_more_heads_than_a_row_has_slots(lib, H, d):
    # a head takes a slot of 8 values however narrow it is, and the kernels hold 2048 slots of a row
    for fn, table in ((lib.gla_join_fwd, JOIN_FWD), (lib.gla_join_bwd, JOIN_BWD)):
        assert call(fn, *table, H=H, d=d) == UN
        assert b"heads are above 2048" in lib.gla_last_error()
    assert lib.gla_join_workspace_size(1, H, 1, d) == 0 and b"heads are above 2048" in lib.gla_last_error()
    for h in (2048, 2047):
        assert lib.gla_join_workspace_size(1, h, 1, d) > 0


def _apart(table):
    """The table with its pointers so far apart that no tensor of the defaults reaches another."""
    names, d = table
    far = dict(d)
    for i, n in enumerate(names):
        if isinstance(d[n], ctypes.c_void_p):
            far[n] = ctypes.c_void_p((i + 1) << 32)
    return names, far


# (call, table, the tensor that is moved, the one it is moved into, bytes from that one's start): the moved
# one's first byte on another's last, or its last byte on another's first
OVERLAPS = [
    ("gla_recur_fwd", RECUR_FWD, "h", "x", 64), ("gla_recur_fwd", RECUR_FWD, "h", "x", 2 * 300 * 64 * 2 - 2),
    ("gla_recur_fwd", RECUR_FWD, "h", "x", -2 * 300 * 64 * 2 + 2), ("gla_recur_fwd", RECUR_FWD, "h", "h0", 508),
    ("gla_recur_fwd", RECUR_FWD, "chunk_in", "h", -2 * 3 * 64 * 4 + 2), ("gla_recur_fwd", RECUR_FWD, "h_final", "g", 4),
    ("gla_recur_fwd", RECUR_FWD, "ws", "g", 2 * 300 * 64 * 4 - 8), ("gla_recur_fwd", RECUR_FWD, "lens", "h_final", 508),
    ("gla_recur_bwd", RECUR_BWD, "dx", "dh", 128), ("gla_recur_bwd", RECUR_BWD, "dg", "chunk_in", 2 * 3 * 64 * 4 - 4),
    ("gla_recur_bwd", RECUR_BWD, "dh0", "dg", 2 * 300 * 64 * 4 - 4), ("gla_recur_bwd", RECUR_BWD, "dhT", "dh0", 508),
    ("gla_recur_bwd", RECUR_BWD, "ws", "lens", -8),
    ("gla_recur_step", RECUR_STEP, "state", "g", -4 * 64 * 4 + 4), ("gla_recur_step", RECUR_STEP, "h", "state", 1020),
    ("gla_recur_step", RECUR_STEP, "slots", "h", 252),
    ("gla_step", STEP, "o", "q", 510), ("gla_step", STEP, "state", "v", -4 * 2 * 64 * 64 * 4 + 4),
    ("gla_step", STEP, "o", "state", 4 * 2 * 64 * 64 * 4 - 2), ("gla_step", STEP, "slots", "state", 8),
    ("gla_join_fwd", JOIN_FWD, "out", "y", 2), ("gla_join_fwd", JOIN_FWD, "out", "residual", 256),
    ("gla_join_fwd", JOIN_FWD, "normed", "out", 2 * 10 * 128 * 2 - 2), ("gla_join_fwd", JOIN_FWD, "w_post", "normed", 16),
    ("gla_join_fwd", JOIN_FWD, "rstd_post", "z", -2 * 10 * 2 * 4 + 4), ("gla_join_fwd", JOIN_FWD, "rstd_pre", "scale", 508),
    ("gla_join_bwd", JOIN_BWD, "dy", "y", 2 * 10 * 128 * 2 - 2), ("gla_join_bwd", JOIN_BWD, "dz", "d_out", 2),
    ("gla_join_bwd", JOIN_BWD, "d_residual", "d_normed", -2), ("gla_join_bwd", JOIN_BWD, "dw_post", "w_post", 252),
    ("gla_join_bwd", JOIN_BWD, "dscale", "w_pre", 508), ("gla_join_bwd", JOIN_BWD, "dw_pre", "dscale", 508),
    ("gla_join_bwd", JOIN_BWD, "ws", "rstd_pre", 76), ("gla_join_bwd", JOIN_BWD, "dy", "ws", 3 * 128 * 4 - 4)]


@pytest.mark.parametrize("name,table,moved,into,by", OVERLAPS, ids=lambda v: str(v) if not isinstance(v, tuple) else "")
def test_an_output_inside_another_tensor_is_refused(lib, name, table, moved, into, by):
    table = _apart(table)
    at = ctypes.c_void_p(table[1][into].value + by)
    assert call(getattr(lib, name), *table, **{moved: at}) == E
    assert b"must not overlap inputs or each other" in lib.gla_last_error()


@pytest.mark.parametrize("st,by", [
    (strides(1 << 20, 0, 64), (1 << 21) + 100),       # inside the second sequence's rows
    (strides(1 << 20, 0, 640), 1280 * 299 + 126),     # on the last element of the first one's last row
    (strides(64, 0, 1 << 20), (299 << 21) + 128),     # token-major: the last token's second sequence
    (strides(1 << 20, 0, 0), 0), (strides(0, 0, 64), 300 * 128 - 2)])
def test_an_output_inside_a_views_rows_is_refused(lib, st, by):
    table = _apart(RECUR_FWD)
    at = ctypes.c_void_p(table[1]["x"].value + by)
    assert call(lib.gla_recur_fwd, *table, x_st=st, h=at) == E
    assert b"must not overlap inputs or each other" in lib.gla_last_error()


def test_python_refuses_host_tensors_and_bad_arguments():
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="device tensors only"):
        gla.gla_recur_fwd(x, x)
    with pytest.raises(ValueError, match="device tensors only"):
        gla.gla_recur_step(x[0], x[0], x[0])
    with pytest.raises(ValueError, match="device tensors only"):
        gla.gla_step(x[None], x[None], x[None], x[None], x)
    with pytest.raises(ValueError, match="device tensors only"):
        gla.gla_join_fwd(x[None])
    with pytest.raises(TypeError, match="torch.Tensor"):
        gla.gla_join_fwd(None)
    with pytest.raises(ValueError, match="with join"):
        gla._join_backward(x, {}, {}, x, None)
    with pytest.raises(ValueError, match="go with join"):
        gla._join_backward(x, {}, None, x, None)


@pytest.mark.gpu
def test_python_refuses_tensors_that_do_not_fit():
    x, g = torch.zeros(2, 30, 8, device="cuda"), torch.zeros(2, 30, 8, device="cuda")
    h, c, _ = gla.gla_recur_fwd(x, g)
    for bad, err in ((dict(x=x[0]), ValueError), (dict(x=x.half()), TypeError), (dict(g=g[:, :5]), ValueError),
                     (dict(g=g.double()), TypeError), (dict(g=g.cpu()), ValueError), (dict(mode="linear"), ValueError),
                     (dict(x=torch.zeros(2, 8, 30, device="cuda").transpose(1, 2)), ValueError),
                     (dict(lens=torch.zeros(2, device="cuda")), TypeError), (dict(h0=torch.zeros(3, 8, device="cuda")), ValueError),
                     (dict(h=x.half()), TypeError), (dict(h=x), gla.GLAError), (dict(chunk_in=c, keep_chunk_states=False), ValueError)):
        with pytest.raises(err):
            gla.gla_recur_fwd(**{"x": x, "g": g, **bad})
    for bad, err in ((dict(dh=x[:, :3]), ValueError), (dict(chunk_in=c[:, :0]), ValueError), (dict(dh=x.bfloat16()), TypeError),
                     (dict(dx=x), gla.GLAError)):
        with pytest.raises(err):
            gla.gla_recur_bwd(**{"x": x, "g": g, "dh": h, "chunk_in": c, **bad})
    st = torch.zeros(1, 8, device="cuda")
    with pytest.raises(ValueError):
        gla.gla_recur_step(x[:, 0], g[:, 0], st)  # 2 rows, 1 state, no slots
    with pytest.raises(TypeError):
        gla.gla_recur_step(x[:, 0], g[:, 0], st, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    y = torch.zeros(1, 2, 5, 16, device="cuda")
    with pytest.raises(ValueError):
        gla.gla_step(y, y, y, y, torch.zeros(1, 2, 16, 8, device="cuda"))
    with pytest.raises(ValueError):
        gla.gla_join_fwd(y, z=torch.zeros(1, 5, 31, device="cuda"))
    with pytest.raises(gla.GLAError):
        gla.gla_join_fwd(y, residual=torch.zeros(1, 5, 32, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gla.gla_join_fwd(y, act="relu")
    with pytest.raises(gla.GLAError):
        gla.gla_join_fwd(y, eps=0.0)
    f = gla.gla_join_fwd(y)
    with pytest.raises(ValueError):
        gla.gla_join_bwd(y, f)
    with pytest.raises(ValueError):
        gla.gla_join_bwd(y, f, d_normed=torch.zeros(1, 5, 32, device="cuda"))
