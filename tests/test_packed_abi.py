"""The packed and norm entry points without a GPU: struct layouts, and every refusal happens on the
host before anything is launched."""
import ctypes

import pytest

import chunked_gated_delta_gdr_amd as G

BASE, MB = 1 << 32, 1 << 26   # fake, aligned, disjoint addresses (never dereferenced)


def at(i):
    return BASE + i * MB


def pdesc(**kw):
    d = dict(n_tokens=100, n_seqs=5, Hk=2, Hv=4, Dk=64, Dv=32, n_slots=8, decay=G.GDR_DECAY_SCALAR)
    d.update(kw)
    return G.make_packed_desc(**d)


def pins(**kw):
    d = dict(q=at(0), k=at(1), v=at(2), beta=at(3), log_alpha=at(4), cu_seqlens=at(5), state_index=at(6),
             has_state=at(7))
    d.update(kw)
    return G.gdr_packed_inputs_t(**d)


def pcheck(expect, d=None, ins=None, pool=at(10), out=at(11), ws=at(12), ws_bytes=MB, for_step=False):
    st = G.gdr_validate_packed(d or pdesc(), ins or pins(), pool, out, ws, ws_bytes, for_step)
    assert st == expect, (st, G.gdr_last_error())
    assert (G.gdr_last_error() != "") == (expect != G.GDR_OK)


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(G.gdr_packed_desc_t) == 12 * 4 + 3 * 4 + 4 + 5 * 8
    assert ctypes.sizeof(G.gdr_packed_inputs_t) == 10 * 8
    assert ctypes.sizeof(G.gdr_norm_desc_t) == 6 * 4 + 4 * 8


def test_valid_packed_calls():
    for step in (False, True):
        pcheck(G.GDR_OK, for_step=step)
        pcheck(G.GDR_OK, ins=pins(state_index=None, has_state=None), for_step=step)
        pcheck(G.GDR_OK, d=pdesc(decay=G.GDR_DECAY_NONE), ins=pins(log_alpha=None), for_step=step)
        pcheck(G.GDR_OK, d=pdesc(n_tokens=0), ins=pins(q=None, k=None, v=None, beta=None, log_alpha=None), out=None,
               for_step=step)
        pcheck(G.GDR_OK, d=pdesc(n_seqs=0), for_step=step)
        pcheck(G.GDR_OK, ins=pins(norm_weight=at(8)), for_step=step)
        pcheck(G.GDR_OK, ins=pins(norm_weight=at(8), norm_gate=at(9)), for_step=step)
        for io in (G.GDR_F32, G.GDR_BF16, G.GDR_F16):
            pcheck(G.GDR_OK, d=pdesc(io_dtype=io), for_step=step)
    pcheck(G.GDR_OK, d=pdesc(n_slots=0), ins=pins(has_state=None), pool=None)
    pcheck(G.GDR_OK, d=pdesc(n_tokens=5), ins=pins(cu_seqlens=None), for_step=True)


@pytest.mark.parametrize("field,value,status", [
    ("struct_size", 4, G.GDR_EINVAL), ("n_tokens", -1, G.GDR_EINVAL), ("n_seqs", -1, G.GDR_EINVAL),
    ("n_seqs", 65536, G.GDR_ENOTSUP), ("Hk", 0, G.GDR_EINVAL), ("Hk", 3, G.GDR_EINVAL), ("Hv", 0, G.GDR_EINVAL),
    ("Hv", 5, G.GDR_EINVAL), ("Hv", 65536, G.GDR_ENOTSUP), ("Dk", 0, G.GDR_EINVAL), ("Dk", 129, G.GDR_ENOTSUP),
    ("Dv", 0, G.GDR_EINVAL), ("Dv", 513, G.GDR_ENOTSUP), ("n_slots", -1, G.GDR_EINVAL), ("io_dtype", 3, G.GDR_EINVAL),
    ("decay", G.GDR_DECAY_CHANNEL, G.GDR_ENOTSUP), ("decay", 7, G.GDR_EINVAL), ("qk_norm", 2, G.GDR_EINVAL),
    ("impl", 3, G.GDR_EINVAL), ("scale", float("nan"), G.GDR_EINVAL), ("qk_eps", -1.0, G.GDR_EINVAL),
    ("norm_eps", float("inf"), G.GDR_EINVAL), ("q_stride", 127, G.GDR_EINVAL), ("k_stride", -5, G.GDR_EINVAL),
    ("v_stride", 1, G.GDR_EINVAL), ("out_stride", 127, G.GDR_EINVAL), ("gate_stride", 127, G.GDR_EINVAL),
    ("n_tokens", 1 << 25, G.GDR_ENOTSUP), ("q_stride", (1 << 23) + 1, G.GDR_ENOTSUP)])
def test_bad_packed_descriptor(field, value, status):
    d = pdesc()
    setattr(d, field, value)
    for step in (False, True):
        pcheck(status, d=d, for_step=step)
    assert G.gdr_packed_fwd_impl(d) == -1 and G.gdr_packed_fwd_workspace_size(d) == 0


def test_packed_pointers():
    for step in (False, True):
        for name in ("q", "k", "v", "beta", "log_alpha"):
            pcheck(G.GDR_EINVAL, ins=pins(**{name: None}), for_step=step)
        pcheck(G.GDR_EINVAL, out=None, for_step=step)
        pcheck(G.GDR_EINVAL, d=pdesc(decay=G.GDR_DECAY_NONE), for_step=step)           # log_alpha without a decay
        pcheck(G.GDR_EINVAL, ins=pins(norm_gate=at(9)), for_step=step)                 # gate without norm
        pcheck(G.GDR_EINVAL, ins=pins(state_index=None), d=pdesc(n_slots=4), for_step=step)
        pcheck(G.GDR_EINVAL, ins=pins(q=at(0) + 1), for_step=step)
        pcheck(G.GDR_EINVAL, ins=pins(cu_seqlens=at(5) + 2), for_step=step)
        pcheck(G.GDR_EINVAL, pool=at(10) + 2, for_step=step)
        # overlaps: a written range with each input, and with each other
        for name in ("q", "k", "v", "beta", "log_alpha", "cu_seqlens", "state_index", "has_state"):
            pcheck(G.GDR_EINVAL, out=getattr(pins(), name), for_step=step)
            pcheck(G.GDR_EINVAL, pool=getattr(pins(), name), for_step=step)
        pcheck(G.GDR_EINVAL, out=at(10), for_step=step)
    pcheck(G.GDR_EINVAL, ins=pins(cu_seqlens=None))
    pcheck(G.GDR_EINVAL, ins=pins(cu_seqlens=None), for_step=True)                     # 100 tokens, 5 sequences
    pcheck(G.GDR_EINVAL, pool=None, d=pdesc(n_slots=0), ins=pins(has_state=None), for_step=True)
    pcheck(G.GDR_EINVAL, pool=None, ins=pins(has_state=None))                          # slots without a pool
    pcheck(G.GDR_EINVAL, pool=None, d=pdesc(n_slots=0))                                # has_state without a pool
    # the last element of a strided out reaches into beta
    far = pdesc(out_stride=(at(3) - at(2)) // 2 // 99)
    pcheck(G.GDR_EINVAL, d=far, out=at(2) + 2 * 4 * 32 * 100, ins=pins(v=at(20)))


def test_packed_workspace():
    d = pdesc(Dk=128, Dv=128)
    need = G.gdr_packed_fwd_workspace_size(d)
    if need:
        pcheck(G.GDR_EINVAL, d=d, ws=None, ws_bytes=0)
        pcheck(G.GDR_EINVAL, d=d, ws_bytes=need - 1)
        pcheck(G.GDR_EINVAL, d=d, ws=at(12) + 64)
        pcheck(G.GDR_EINVAL, d=d, ws=at(11))
        pcheck(G.GDR_OK, d=d, ws_bytes=need)
    d = pdesc(Dk=128, Dv=128, impl=G.GDR_IMPL_GENERIC)
    assert G.gdr_packed_fwd_workspace_size(d) == 0
    pcheck(G.GDR_OK, d=d, ws=None, ws_bytes=0)
    assert G.gdr_packed_fwd_impl(pdesc(Dk=100, impl=G.GDR_IMPL_MFMA)) == -1
    assert G.gdr_packed_fwd_impl(pdesc(Dk=100)) == G.GDR_IMPL_GENERIC


def ncheck(expect, d, **kw):
    p = dict(x=at(0), y=at(1))
    p.update(kw)
    st = G.gdr_validate_norm(d, **p)
    assert st == expect, (st, G.gdr_last_error())


def test_norm_arguments():
    d = G.make_norm_desc(rows=10, D=128)
    ncheck(G.GDR_OK, d)
    ncheck(G.GDR_OK, d, y=at(0))                                                       # in place
    ncheck(G.GDR_OK, d, weight=at(2), gate=at(3), residual=at(4), residual_out=at(5))
    ncheck(G.GDR_OK, d, residual=at(4), residual_out=at(4))
    ncheck(G.GDR_OK, d, residual=at(4), residual_out=at(0))
    ncheck(G.GDR_EINVAL, d, y=at(0), residual=at(4), residual_out=at(5))               # y on x beside a residual
    ncheck(G.GDR_EINVAL, d, y=at(0) + 256)                                             # shifted
    ncheck(G.GDR_EINVAL, d, residual=at(4))
    ncheck(G.GDR_EINVAL, d, residual_out=at(4))
    ncheck(G.GDR_EINVAL, d, residual=at(4), residual_out=at(1))                        # the sum on y
    ncheck(G.GDR_EINVAL, d, residual=at(1), residual_out=at(5))                        # y on residual
    ncheck(G.GDR_EINVAL, d, scales=at(6))
    ncheck(G.GDR_EINVAL, d, x=None)
    ncheck(G.GDR_EINVAL, d, y=None)
    ncheck(G.GDR_EINVAL, d, x=at(0) + 1)
    ncheck(G.GDR_EINVAL, d, weight=at(1))
    ncheck(G.GDR_EINVAL, d, gate=at(1))
    wide = G.make_norm_desc(rows=10, D=128, x_stride=256)
    ncheck(G.GDR_OK, wide)
    ncheck(G.GDR_EINVAL, wide, y=at(0))                                                # in place over strided rows
    codes = G.make_norm_desc(rows=10, D=128, out_kind=G.GDR_OUT_INT8)
    ncheck(G.GDR_EINVAL, codes)
    ncheck(G.GDR_OK, codes, scales=at(6))
    ncheck(G.GDR_OK, codes, scales=at(6), y=at(1) + 1)                                 # bytes need no alignment
    ncheck(G.GDR_EINVAL, codes, scales=at(6), y=at(0))
    ncheck(G.GDR_EINVAL, codes, scales=at(0))
    ncheck(G.GDR_EINVAL, codes, scales=at(1))
    ncheck(G.GDR_OK, G.make_norm_desc(rows=0, D=128), x=None, y=None)


@pytest.mark.parametrize("field,value,status", [
    ("struct_size", 4, G.GDR_EINVAL), ("rows", -1, G.GDR_EINVAL), ("D", 0, G.GDR_EINVAL), ("D", 16385, G.GDR_ENOTSUP),
    ("io_dtype", 5, G.GDR_EINVAL), ("out_kind", 3, G.GDR_EINVAL), ("eps", -1.0, G.GDR_EINVAL),
    ("eps", float("nan"), G.GDR_EINVAL), ("x_stride", 127, G.GDR_EINVAL), ("residual_stride", -1, G.GDR_EINVAL),
    ("gate_stride", 5, G.GDR_EINVAL), ("dy_stride", 5, G.GDR_EINVAL), ("rows", 2 ** 31 - 1, G.GDR_ENOTSUP)])
def test_bad_norm_descriptor(field, value, status):
    d = G.make_norm_desc(rows=10, D=128)
    setattr(d, field, value)
    ncheck(status, d)
    assert G.gdr_validate_norm_bwd(d, at(0), at(1), dx=at(2)) == status
    assert G.gdr_rms_norm_bwd_workspace_size(d) == 0


def test_norm_bwd_arguments():
    d = G.make_norm_desc(rows=10, D=128)
    need = G.gdr_rms_norm_bwd_workspace_size(d)
    assert need >= 128 * 4

    def check(expect, **kw):
        p = dict(x=at(0), dy=at(1), dx=at(2))
        p.update(kw)
        st = G.gdr_validate_norm_bwd(d, **p)
        assert st == expect, (st, G.gdr_last_error())
    ws = dict(dweight=at(3), workspace=at(4), workspace_bytes=need)
    check(G.GDR_OK)
    check(G.GDR_OK, weight=at(5), gate=at(6), dgate=at(7), d_residual=at(8), **ws)
    for name in ("x", "dy", "dx"):
        check(G.GDR_EINVAL, **{name: None})
    check(G.GDR_EINVAL, gate=at(6))
    check(G.GDR_EINVAL, dgate=at(6))
    check(G.GDR_EINVAL, dx=at(1))
    check(G.GDR_EINVAL, d_residual=at(2))
    check(G.GDR_EINVAL, dweight=at(3))
    check(G.GDR_EINVAL, **dict(ws, workspace_bytes=need - 1))
    check(G.GDR_EINVAL, **dict(ws, workspace=at(4) + 8))
    check(G.GDR_EINVAL, **dict(ws, workspace=at(2)))
    check(G.GDR_EINVAL, **dict(ws, dweight=at(3) + 2))
    codes = G.make_norm_desc(rows=10, D=128, out_kind=G.GDR_OUT_FP8)
    assert G.gdr_validate_norm_bwd(codes, at(0), at(1), dx=at(2)) == G.GDR_ENOTSUP


def test_cpu_tensors_are_refused():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        G.gdr_rms_norm(x)
    with pytest.raises(ValueError):
        G.gdr_rms_norm_bwd(x, x)
    q = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        G.gdr_packed_step(q, q, q, torch.zeros(4, 2, 8, 8), beta=torch.zeros(4, 2))
    with pytest.raises(ValueError):
        G.gdr_packed_fwd(q, q, q, torch.zeros(2, dtype=torch.int32), beta=torch.zeros(4, 2))


def test_most_rows_of_a_packed_call():
    """n_tokens * Hv: 2^26 is the last that both take, with the output norm's launch too."""
    ins = pins(norm_weight=at(8), q=1 << 40, k=1 << 41, v=1 << 42, beta=1 << 43, log_alpha=1 << 44)
    for step in (False, True):
        d = pdesc(n_tokens=1 << 21, Hk=1, Hv=32, Dk=8, Dv=8)
        pcheck(G.GDR_OK, d=d, ins=ins, out=1 << 45, ws=1 << 46, ws_bytes=1 << 40, for_step=step)
        d.n_tokens += 1
        pcheck(G.GDR_ENOTSUP, d=d, ins=ins, out=1 << 45, ws=1 << 46, ws_bytes=1 << 40, for_step=step)


def test_arguments_by_name():
    """Every tensor may be named, the first too, and the signatures say that a stream may be given."""
    import inspect
    import torch
    q = torch.zeros(4, 2, 8)
    cu = torch.zeros(2, dtype=torch.int32)
    calls = [(G.gdr_packed_fwd, dict(q=q, k=q, v=q, cu_seqlens=cu, beta=q[..., 0])),
             (G.gdr_packed_step, dict(q=q, k=q, v=q, state=torch.zeros(4, 2, 8, 8), beta=q[..., 0])),
             (G.gdr_rms_norm, dict(x=q[0])), (G.gdr_rms_norm_bwd, dict(x=q[0], dy=q[0]))]
    for call, kw in calls:
        with pytest.raises(ValueError, match="must be on a GPU"):
            call(**kw)
        first = next(iter(kw))
        with pytest.raises(TypeError, match=f"'{first}'"):
            call(**{n: t for n, t in kw.items() if n != first})
        stream = inspect.signature(call).parameters["stream"]
        assert stream.kind is inspect.Parameter.KEYWORD_ONLY and stream.default is None
        assert list(inspect.signature(call).parameters)[0] == first
