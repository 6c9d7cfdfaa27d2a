"""The gated delta rule's and the layer norm's calls without a GPU: every refusal happens on the host, before any HIP
call."""
import ctypes

import pytest
import torch

from sequence_state_scan_amd import gla

E, UN = gla.GLA_ERR_INVALID_ARG, gla.GLA_ERR_UNSUPPORTED


def p(i):
    return ctypes.c_void_p((i + 1) << 32)  # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    return gla.load_library()


def strides(*v):
    return (ctypes.c_longlong * 3)(*v)


def table(text, **ints):
    """Names in order and their defaults: pointers apart from each other, strides NULL, numbers as given."""
    names = text.split()
    d = {n: ints[n] if n in ints else None if n.endswith("_st") or n == "stream" else p(i) for i, n in enumerate(names)}
    return names, d


IN = "q q_st k k_st v v_st g g_st beta b_st "
FWD = table(IN + "h0 lens o h_final saved saved_size B H Hk T dk dv dtype ws wsb stream", B=2, H=4, Hk=2, T=300, dk=64, dv=96,
            dtype=1, saved_size=1 << 31, wsb=1 << 31)
BWD = table(IN + "o do do_st saved saved_size lens dhT dq dk_ dv_ dg dbeta dh0 B H Hk T dk dv dtype ws wsb stream", B=2, H=4,
            Hk=2, T=300, dk=64, dv=96, dtype=1, saved_size=1 << 31, wsb=1 << 31)
STEP = table(IN + "state slots o B H Hk n dk dv n_slots dtype stream", B=2, H=4, Hk=2, n=1, dk=64, dv=96, n_slots=4, dtype=1)
NORM = table("x x_st residual r_st w b out normed mean rstd B T D eps dtype stream_dtype stream", B=2, T=10, D=64, eps=1e-5,
             dtype=1, stream_dtype=1)
NORM_BWD = table("x x_st residual r_st w mean rstd d_out do_st d_normed dn_st dx d_residual dw db B T D dtype stream_dtype ws "
                 "wsb stream", B=2, T=10, D=64, dtype=1, stream_dtype=1, wsb=1 << 30)


def call(fn, tab, **kw):
    names, d = tab
    assert not set(kw) - set(names), kw
    return fn(*[kw.get(n, d[n]) for n in names])


def off(v, by):
    return ctypes.c_void_p(v.value + by)


SIZES = [(dict(B=0), E), (dict(H=0), E), (dict(Hk=0), E), (dict(T=0), E), (dict(dk=0), E), (dict(dv=-1), E), (dict(Hk=3), E),
         (dict(dtype=2), E), (dict(dk=129), UN), (dict(dv=1025), UN), (dict(B=1 << 12, H=1 << 10), UN),
         (dict(B=64, H=64, T=1 << 17), UN)]
INPUTS = [(dict(q=None), E), (dict(k=None), E), (dict(v=None), E), (dict(g=None), E), (dict(beta=None), E),
          (dict(q_st=strides(-1, 0, 64)), E), (dict(g_st=strides(0, 0, -1)), E), (dict(b_st=strides(0, -1, 1)), E)]


@pytest.mark.parametrize("kw,want", SIZES + INPUTS + [
    (dict(o=None), E), (dict(ws=None), E), (dict(wsb=64), E), (dict(saved_size=64), E), (dict(ws=ctypes.c_void_p(8 + (50 << 32))), E),
    (dict(saved=ctypes.c_void_p(4 + (60 << 32))), E), (dict(o=p(0)), E), (dict(h_final=FWD[1]["h0"]), E),
    (dict(saved=FWD[1]["o"]), E), (dict(ws=FWD[1]["saved"]), E), (dict(o=off(FWD[1]["g"], 2 * 4 * 300 * 4 - 2)), E),
    (dict(h_final=off(FWD[1]["lens"], -2 * 4 * 64 * 96 * 4 + 4)), E)])
def test_delta_fwd_refusals(lib, kw, want):
    assert call(lib.gla_delta_fwd, FWD, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_delta_fwd: ")


@pytest.mark.parametrize("kw,want", SIZES + INPUTS + [
    (dict(o=None), E), (dict(do=None), E), (dict(saved=None), E), (dict(dq=None), E), (dict(dk_=None), E), (dict(dv_=None), E),
    (dict(dg=None), E), (dict(dbeta=None), E), (dict(ws=None), E), (dict(wsb=64), E), (dict(saved_size=64), E),
    (dict(do_st=strides(0, 0, -1)), E), (dict(dq=p(0)), E), (dict(dv_=BWD[1]["do"]), E), (dict(dg=BWD[1]["dbeta"]), E),
    (dict(dh0=BWD[1]["dhT"]), E), (dict(ws=BWD[1]["saved"]), E), (dict(dk_=BWD[1]["o"]), E)])
def test_delta_bwd_refusals(lib, kw, want):
    assert call(lib.gla_delta_bwd, BWD, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_delta_bwd: ")


@pytest.mark.parametrize("kw,want", INPUTS + [
    (dict(B=0), E), (dict(n=0), E), (dict(Hk=3), E), (dict(dtype=7), E), (dict(dk=257), UN), (dict(state=None), E), (dict(o=None), E),
    (dict(slots=None, n_slots=1), E), (dict(n_slots=0), E), (dict(state=p(0)), E), (dict(o=STEP[1]["beta"]), E),
    (dict(B=1 << 20, H=1 << 10, n_slots=1 << 21), UN)])
def test_delta_step_refusals(lib, kw, want):
    assert call(lib.gla_delta_step, STEP, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_delta_step: ")


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), E), (dict(T=0), E), (dict(D=0), E), (dict(D=16385), UN), (dict(dtype=3), E), (dict(stream_dtype=3), E),
    (dict(dtype=0, stream_dtype=1), UN), (dict(x=None), E), (dict(normed=None), E), (dict(residual=None), E), (dict(mean=None), E),
    (dict(rstd=None), E), (dict(eps=0.0), E), (dict(eps=float("nan")), E), (dict(x_st=strides(-1, 0, 0)), E),
    (dict(out=NORM[1]["x"]), E), (dict(normed=NORM[1]["residual"]), E), (dict(mean=NORM[1]["w"]), E),
    (dict(out=NORM[1]["residual"], r_st=strides(1280, 0, 128)), E)])
def test_layernorm_fwd_refusals(lib, kw, want):
    assert call(lib.gla_layernorm_fwd, NORM, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_layernorm_fwd: ")


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), E), (dict(D=16385), UN), (dict(dtype=0, stream_dtype=1), UN), (dict(x=None), E), (dict(mean=None), E),
    (dict(rstd=None), E), (dict(d_normed=None), E), (dict(dx=None), E), (dict(residual=None), E), (dict(ws=None), E),
    (dict(wsb=16), E), (dict(ws=ctypes.c_void_p(2 + (50 << 32))), E), (dict(dx=NORM_BWD[1]["x"]), E),
    (dict(dw=NORM_BWD[1]["db"]), E), (dict(d_residual=NORM_BWD[1]["d_out"]), E), (dict(do_st=strides(0, 0, -1)), E)])
def test_layernorm_bwd_refusals(lib, kw, want):
    assert call(lib.gla_layernorm_bwd, NORM_BWD, **kw) == want
    assert lib.gla_last_error().startswith(b"gla_layernorm_bwd: ")


def test_sizes(lib):
    dims = (1, 2, 1, 5000, 64, 64)
    for which in (gla.GLA_FWD, gla.GLA_BWD):
        assert gla.delta_workspace_size(which, *dims, torch.bfloat16) > 0
    assert lib.gla_delta_workspace_size(2, *dims, 1) == 0 and lib.gla_last_error()
    assert lib.gla_delta_saved_size(1, 3, 2, 5, 5, 5, 0) == 0 and b"multiple" in lib.gla_last_error()
    with pytest.raises(gla.GLAError):
        gla.delta_saved_size(1, 2, 1, 5, 200, 64, torch.float32)
    with pytest.raises(gla.GLAError):
        gla.layernorm_workspace_size(1, 1, 0)
    assert gla.layernorm_workspace_size(1, 1, 100) >= 2 * 100 * 4


def test_python_calls_refuse_what_is_not_on_a_gpu():
    q, g = torch.zeros(1, 1, 4, 8), torch.zeros(1, 1, 4)
    with pytest.raises(ValueError, match="device tensors"):
        gla.gla_delta_fwd(q, q, q, g, g)
    with pytest.raises(ValueError, match="device tensors"):
        gla.gla_delta_step(q, q, q, g, g, torch.zeros(1, 1, 8, 8))
    with pytest.raises(ValueError, match="device tensors"):
        gla.gla_layernorm_fwd(torch.zeros(1, 2, 8))
    with pytest.raises(TypeError, match="torch.Tensor"):
        gla.gla_layernorm_fwd(None)
