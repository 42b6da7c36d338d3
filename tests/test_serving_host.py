"""The serving entry points on the host (no GPU): what the C ABI and the
binding refuse before anything is launched, and the cache's layout."""
import ctypes

import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNCore, GDNStateCache

P = ctypes.c_void_p(256)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p(264)
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


def shape(**kw):
    base = dict(n_seq=2, total_tokens=3, hk=2, hv=6, d=128, dtype=L.GDN_BF16)
    base.update(kw)
    return L.make_shape(base["n_seq"], base["total_tokens"], base["hk"], base["hv"], base["d"], base["dtype"])


def cache(**kw):
    base = dict(S_ptr=256, S_stride=6 * 128 * 128, conv_ptr=256, conv_stride=3 * 1280, n_slots=5)
    base.update(kw)
    return L.Cache(*base.values())


def rule(sh=None, c=None, **kw):
    a = dict(q=P, k=P, v=P, ldq=256, ldk=256, ldv=768, g=P, beta=P, cu=P, o=P)
    a.update(kw)
    sh = shape() if sh is None else sh
    return L.load().gdn_recurrent_fwd(
        ctypes.byref(sh), a["q"], a["k"], a["v"], a["ldq"], a["ldk"], a["ldv"], a["g"], a["beta"], 0.1,
        ctypes.byref(cache() if c is None else c), None, None, None, a["cu"], a["o"], None)


def step(sh=None, c=None, **kw):
    a = dict(x=P, ldx=1280, w=P, a=P, lda=6, b=P, ldb=6, A=P, dt=P, z=P, ldz=768, wn=P, l2=1e-6, ne=1e-6,
             act=0, cu=P, out=P)
    a.update(kw)
    sh = shape() if sh is None else sh
    return L.load().gdn_step_fwd(
        ctypes.byref(sh), a["x"], a["ldx"], a["w"], a["a"], a["lda"], a["b"], a["ldb"], a["A"], a["dt"],
        a["z"], a["ldz"], a["wn"], 0.1, a["l2"], a["ne"], a["act"],
        ctypes.byref(cache() if c is None else c), None, None, None, a["cu"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(g=None), INVALID), (dict(beta=None), INVALID), (dict(cu=None), INVALID),
    (dict(q=ODD), ALIGNMENT), (dict(o=ODD), ALIGNMENT), (dict(ldq=255), INVALID), (dict(ldk=260), ALIGNMENT),
    (dict(ldv=760), INVALID), (dict(sh=shape(d=64)), UNSUPPORTED), (dict(sh=shape(hv=5)), INVALID),
    (dict(sh=shape(n_seq=0)), INVALID), (dict(sh=shape(total_tokens=-1)), INVALID),
    (dict(c=cache(S_ptr=None)), INVALID), (dict(c=cache(n_slots=0)), INVALID),
    (dict(c=cache(S_stride=6 * 128 * 128 - 4)), INVALID), (dict(c=cache(S_stride=6 * 128 * 128 + 2)), ALIGNMENT),
    (dict(c=cache(S_ptr=260)), ALIGNMENT)])
def test_rule_refusals(kw, status):
    assert rule(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID),
    (dict(A=None), INVALID), (dict(dt=None), INVALID), (dict(z=None), INVALID), (dict(wn=None), INVALID),
    (dict(cu=None), INVALID), (dict(out=None), INVALID), (dict(x=ODD), ALIGNMENT), (dict(z=ODD), ALIGNMENT),
    (dict(ldx=1272), INVALID), (dict(ldx=1284), ALIGNMENT), (dict(ldz=760), INVALID), (dict(ldz=772), ALIGNMENT),
    (dict(lda=5), INVALID), (dict(ldb=5), INVALID), (dict(l2=-1.0), INVALID), (dict(ne=-1.0), INVALID),
    (dict(ne=float("nan")), INVALID), (dict(act=2), INVALID), (dict(sh=shape(d=64)), UNSUPPORTED),
    (dict(c=cache(conv_ptr=None)), INVALID), (dict(c=cache(conv_stride=3 * 1280 - 8)), INVALID),
    (dict(c=cache(conv_ptr=264)), ALIGNMENT), (dict(c=cache(conv_stride=3 * 1280 + 4)), ALIGNMENT),
    (dict(c=cache(S_ptr=None)), INVALID)])
def test_step_refusals(kw, status):
    assert step(**kw) == status


def test_null_cache_is_refused():
    lib, sh = L.load(), shape()
    assert lib.gdn_recurrent_fwd(ctypes.byref(sh), P, P, P, 256, 256, 768, P, P, 0.1, None, None, None, None, P,
                                 P, None) == INVALID


def test_check_slots_refusals():
    f, sh = L.load().gdn_check_slots, shape()
    assert f(ctypes.byref(sh), 0, P, P, P, P, P, None) == INVALID
    assert f(ctypes.byref(sh), 4, P, P, P, None, P, None) == INVALID
    assert f(ctypes.byref(sh), 4, P, P, P, P, None, None) == INVALID
    assert f(ctypes.byref(sh), 4, P, P, P, P, ctypes.c_void_p(258), None) == ALIGNMENT
    assert f(ctypes.byref(shape(n_seq=0)), 4, P, P, P, P, P, None) == INVALID


def test_cache_refusals():
    lib = L.load()
    n = lib.gdn_cache_workspace(5)
    assert n >= 16 + 2 * 4 * 5 and lib.gdn_cache_workspace(0) == 0
    copy, fork, compact = lib.gdn_cache_copy, lib.gdn_cache_fork, lib.gdn_cache_compact
    for args, st in (((None, 32, 5, P, P, 32, 5, P, 32, 1), INVALID), ((P, 32, 5, P, None, 32, 5, P, 32, 1), INVALID),
                     ((P, 32, 0, P, P, 32, 5, P, 32, 1), INVALID), ((P, 32, 5, P, P, 32, 5, P, 32, -1), INVALID),
                     ((P, 16, 5, P, P, 32, 5, P, 32, 1), INVALID), ((P, 32, 5, P, P, 32, 5, P, -16, 1), INVALID),
                     ((P, 40, 5, P, P, 32, 5, P, 32, 1), ALIGNMENT), ((P, 32, 5, P, P, 32, 5, P, 24, 1), ALIGNMENT),
                     ((ODD, 32, 5, P, P, 32, 5, P, 32, 1), ALIGNMENT), ((P, 32, 5, P, P, 32, 5, P, 32, 0), OK)):
        assert copy(*args, None) == st, args
    for args, st in (((None, 32, 5, P, P, 1, P, P, n), INVALID), ((P, 32, 5, None, P, 1, P, P, n), INVALID),
                     ((P, 32, 5, P, None, 1, P, P, n), INVALID), ((P, 32, 5, P, P, 1, None, P, n), INVALID),
                     ((P, 32, 5, P, P, -1, P, P, n), INVALID), ((P, 24, 5, P, P, 1, P, P, n), ALIGNMENT),
                     ((P, 32, 5, P, P, 1, P, None, n), WORKSPACE), ((P, 32, 5, P, P, 1, P, P, n - 1), WORKSPACE),
                     ((P, 32, 5, P, P, 1, P, ODD, n), WORKSPACE), ((P, 32, 5, P, None, 0, None, P, n), OK)):
        assert fork(*args, None) == st, args
    for args, st in (((None, 32, 5, P, P, P, 1, P, n), INVALID), ((P, 32, 5, None, P, P, 1, P, n), INVALID),
                     ((P, 32, 5, P, None, P, 1, P, n), INVALID), ((P, 32, 5, P, P, None, 1, P, n), INVALID),
                     ((P, 32, 5, P, P, P, -1, P, n), INVALID), ((P, 32, 0, P, P, P, 1, P, n), INVALID),
                     ((P, 32, 5, P, P, P, 1, P, n - 1), WORKSPACE)):
        assert compact(*args, None) == st, args
    for f in (lib.gdn_cache_retain, lib.gdn_cache_release):
        assert f(None, 5, P, 1, None) == INVALID and f(P, 0, P, 1, None) == INVALID
        assert f(P, 5, None, 1, None) == INVALID and f(P, 5, P, -1, None) == INVALID
        assert f(P, 5, None, 0, None) == OK


def test_make_cache_checks_the_views():
    S, conv = torch.zeros(3, 4, 32, 32), torch.zeros(3, 3, 256, dtype=torch.bfloat16)
    c = L.make_cache(S, conv)
    assert (c.n_slots, c.S_stride, c.conv_stride, c.heads) == (3, 4096, 768, (4, 32))
    for bad in (S.half(), S[0], S.transpose(2, 3), S[:, :, :16], torch.zeros(0, 4, 32, 32)):
        with pytest.raises(ValueError):
            L.make_cache(bad, conv)
    for bad in (conv.double(), conv[:2], conv[:, :2], conv[:, :, ::2]):
        with pytest.raises(ValueError):
            L.make_cache(S, bad)


def test_the_binding_checks_its_arguments():
    """Each case breaks one argument; a correct host call is refused as such."""
    sh, T, N = shape(hk=1, hv=2, d=32), 3, 2
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(x=torch.zeros(T, 128, dtype=bf), w_conv=torch.zeros(128, 4), a=torch.zeros(T, 2, dtype=bf),
                b=torch.zeros(T, 2, dtype=bf), A_log=torch.zeros(2), dt_bias=torch.zeros(2),
                z=torch.zeros(T, 64, dtype=bf), w_norm=torch.zeros(32), scale=1.0,
                cache=L.make_cache(torch.zeros(4, 2, 32, 32), torch.zeros(4, 3, 128, dtype=bf)),
                slot_in=torch.zeros(N, dtype=i32), slot_out=None, slot_tok=torch.zeros(T, dtype=i32),
                cu_seqlens=torch.zeros(N + 1, dtype=i32), out=torch.zeros(T, 2, 32, dtype=bf))
    with pytest.raises(ValueError, match="host tensor"):
        L.gdn_step_fwd(sh, **good)
    for name, bad, err in (
            ("x", good["x"].float(), TypeError), ("x", good["x"][:, ::2], ValueError), ("x", good["x"][:2], ValueError),
            ("w_conv", torch.zeros(128, 3), ValueError), ("a", good["a"][:, :1], ValueError),
            ("b", good["b"].float(), TypeError), ("A_log", torch.zeros(3), ValueError),
            ("dt_bias", torch.zeros(2, dtype=bf), TypeError), ("z", torch.zeros(T, 63, dtype=bf), ValueError),
            ("w_norm", torch.zeros(31), ValueError), ("slot_in", torch.zeros(N), TypeError),
            ("slot_in", torch.zeros(N + 1, dtype=i32), ValueError), ("slot_in", torch.zeros(2 * N, dtype=i32)[::2], ValueError),
            ("slot_out", torch.zeros(1, dtype=i32), ValueError), ("slot_tok", torch.zeros(N, dtype=i32), ValueError),
            ("cu_seqlens", torch.zeros(N, dtype=i32), ValueError), ("out", torch.zeros(T, 64), TypeError),
            ("out", torch.zeros(T, 32, dtype=bf), ValueError),
            ("cache", L.make_cache(torch.zeros(4, 1, 32, 32), torch.zeros(4, 3, 128, dtype=bf)), ValueError),
            ("cache", L.make_cache(torch.zeros(4, 2, 32, 32)), ValueError),
            ("cache", L.make_cache(torch.zeros(4, 2, 32, 32), torch.zeros(4, 3, 128)), ValueError),
            ("cache", L.make_cache(torch.zeros(4, 2, 32, 32), torch.zeros(4, 3, 136, dtype=bf)), ValueError)):
        with pytest.raises(err):
            L.gdn_step_fwd(sh, **dict(good, **{name: bad}))


def test_a_tensor_on_another_device_is_refused():
    sh = shape(hk=1, hv=2, d=32, total_tokens=1, n_seq=1)
    c = L.make_cache(torch.zeros(4, 2, 32, 32))
    t = torch.zeros(1, 32, dtype=torch.bfloat16)
    v, f, cu = torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(1, 2), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="k is on meta"):
        L.gdn_recurrent_fwd(sh, t, t.to("meta"), v, f, f, 1.0, c, None, None, None, cu, v)
    with pytest.raises(ValueError, match="slot_in is on meta"):
        L.gdn_recurrent_fwd(sh, t, t, v, f, f, 1.0, c, torch.zeros(1, dtype=torch.int32, device="meta"), None, None,
                            cu, v)


def test_cache_tensors_are_checked():
    buf, refs = torch.zeros(4, 32, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    ws, i2 = torch.zeros(256, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: L.gdn_cache_fork(buf[:, ::2], refs, i2, i2, ws), lambda: L.gdn_cache_fork(buf, refs[:3], i2, i2, ws),
                 lambda: L.gdn_cache_fork(buf, refs, i2, i2[:1], ws), lambda: L.gdn_cache_fork(buf, refs, i2, i2, ws.int()),
                 lambda: L.gdn_cache_compact(buf, refs, i2, None, ws), lambda: L.gdn_cache_copy(buf, buf[:, :16], i2, i2),
                 lambda: L.gdn_cache_copy(buf, buf, i2, i2[:1]), lambda: L.gdn_cache_copy(buf, buf[:3]),
                 lambda: L.gdn_cache_copy(buf, buf[:1], src_idx=i2), lambda: L.gdn_cache_copy(buf[:1], buf, dst_idx=i2),
                 lambda: L.gdn_cache_copy(buf[0], buf, i2, i2), lambda: L.gdn_cache_copy(buf.t(), buf.t(), i2, i2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.gdn_cache_retain(refs, i2.long())
    with pytest.raises(ValueError, match="host tensor"):
        L.gdn_cache_release(refs, i2)


def test_state_cache_layout():
    """Views of all layers' states lie in the buffer without touching."""
    for dt, E in ((torch.bfloat16, 2), (torch.float32, 4)):
        cfg = CoreConfig(1, 2, 32, dt)
        c = GDNStateCache(cfg, 5, n_layers=3, device="cpu")
        assert c.slot_bytes % 256 == 0 and c.buffer.shape == (5, c.slot_bytes) and c.refs.tolist() == [0] * 5
        c.buffer.zero_()
        for k in range(3):
            assert c.S(k).shape == (5, 2, 32, 32) and c.conv(k).shape == (5, 3, 128) and c.conv(k).dtype == dt
            assert c.layer(k).S_ptr % 16 == 0 and c.layer(k).conv_ptr % 16 == 0
            assert c.layer(k).S_stride * 4 == c.layer(k).conv_stride * E == c.slot_bytes
            c.S(k).fill_(k + 1)
            c.conv(k).fill_(k + 11)
        for k in range(3):
            assert bool((c.S(k) == k + 1).all()) and bool((c.conv(k) == k + 11).all())
    buf = torch.zeros(5, c.slot_bytes, dtype=torch.uint8)
    assert GDNStateCache(cfg, 5, 3, "cpu", buffer=buf).buffer is buf
    for kw in (dict(buffer=buf[:4]), dict(buffer=buf.int()), dict(buffer=buf, refs=torch.zeros(4, dtype=torch.int32)),
               dict(refs=torch.zeros(5))):
        with pytest.raises(ValueError):
            GDNStateCache(cfg, 5, 3, "cpu", **kw)
    for n, k in ((0, 1), (1, 0)):
        with pytest.raises(ValueError):
            GDNStateCache(cfg, n, k, "cpu")


def test_prefill_wants_a_slot_for_every_sequence():
    core = GDNCore(CoreConfig(1, 2, 32, torch.bfloat16), "cpu")
    c = GDNStateCache(core.cfg, 4, device="cpu")
    bf = torch.bfloat16
    x, h, z = torch.zeros(3, 128, dtype=bf), torch.zeros(3, 2, dtype=bf), torch.zeros(3, 2, 32, dtype=bf)
    cu = torch.tensor([0, 1, 3], dtype=torch.int32)
    two, one = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for si, so in ((one, two), (two, one), (one, None)):
        with pytest.raises(ValueError, match="2 sequences"):
            core.prefill(x, torch.zeros(128, 4), h, h, torch.zeros(2), torch.zeros(2), z, torch.zeros(32), cu, c, si, so)


def test_core_step_refuses_host_tensors():
    core = GDNCore(CoreConfig(1, 2, 32, torch.bfloat16), "cpu")
    c = GDNStateCache(core.cfg, 2, device="cpu")
    bf = torch.bfloat16
    x, h, z = torch.zeros(1, 128, dtype=bf), torch.zeros(1, 2, dtype=bf), torch.zeros(1, 2, 32, dtype=bf)
    one, cu = torch.zeros(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    with pytest.raises(ValueError, match="host tensor"):
        core.step(x, torch.zeros(128, 4), h, h, torch.zeros(2), torch.zeros(2), z, torch.zeros(32), cu, c, one)
