"""CPU-only checks of the C ABI: the library loads, exports every function the
header declares, and rejects bad arguments before launching anything (these
calls validate on the host and never reach a kernel)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ulysses.h")


@pytest.fixture(scope="module")
def L():
    from long_context_sequence_all_b200 import build, ulysses
    build.build()
    return ulysses.lib()


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ulysses_\w+)\s*\(", text)))


def test_header_declares_the_five_path_entry_points():
    names = declared_functions()
    for n in ["ulysses_seq_to_head", "ulysses_attn_fwd", "ulysses_attn_bwd", "ulysses_head_to_seq",
              "ulysses_loss_aggregate"]:
        assert n in names


def test_library_exports_every_declared_symbol(L):
    for name in declared_functions():
        assert hasattr(L, name), name
    from long_context_sequence_all_b200 import ulysses
    assert set(ulysses.EXPORTS) <= set(declared_functions())


def test_status_strings(L):
    from long_context_sequence_all_b200 import ulysses
    for code, name in ulysses.STATUS.items():
        assert ulysses.ulysses_status_string(code)
    assert ulysses.ulysses_status_string(0) == "ok"


def test_permute_validation(L):
    vp = ctypes.c_void_p
    a, b = vp(1 << 20), vp(1 << 30)   # never dereferenced: validation fails first
    assert L.ulysses_seq_to_head(1, 1024, 4, 8, 64, 4, None, b, None) == 1        # NULL
    assert L.ulysses_seq_to_head(1, 1022, 4, 8, 64, 4, a, b, None) == 2           # n % P
    assert L.ulysses_seq_to_head(1, 1024, 4, 6, 64, 4, a, b, None) == 2           # heads % P
    assert L.ulysses_seq_to_head(1, 1024, 4, 8, 64, 3, a, b, None) == 3           # elem bytes
    assert L.ulysses_seq_to_head(1, 1024, 4, 8, 6, 2, a, b, None) == 4            # row not 16 B
    assert L.ulysses_seq_to_head(1, 1024, 4, 8, 64, 4, vp((1 << 20) + 4), b, None) == 4  # misaligned
    assert L.ulysses_head_to_seq(1, 1024, 4, 8, 64, 4, a, vp((1 << 20) + 4096), None) == 5  # overlap
    assert L.ulysses_seq_to_head(0, 1024, 4, 8, 64, 4, a, b, None) == 2


def test_kv_copy_validation(L):
    vp = ctypes.c_void_p
    a, b = vp(1 << 20), vp(1 << 30)
    rep, red = L.ulysses_kv_seq_to_head_replicated, L.ulysses_kv_head_to_seq_reduce
    assert rep(1, 1024, 8, 2, 128, 2, None, b, None) == 1                 # NULL
    assert rep(1, 1024, 8, 3, 128, 2, a, b, None) == 2                    # P % G
    assert rep(1, 1020, 8, 2, 128, 2, a, b, None) == 2                    # n % P
    assert rep(1, 1024, 8, 2, 128, 3, a, b, None) == 3                    # elem bytes
    assert rep(1, 1024, 8, 2, 4, 2, a, b, None) == 4                      # row not 16 B
    # the copies (dst, P rows per position) overlap a source placed inside them
    assert rep(1, 1024, 8, 2, 128, 2, vp((1 << 20) + 1024 * 2 * 256), a, None) == 5
    assert red(1, 1024, 8, 2, 128, 7, a, b, None) == 3                    # dtype
    assert red(1, 1024, 8, 3, 128, 1, a, b, None) == 2
    assert red(1, 1024, 8, 2, 128, 1, a, vp((1 << 20) + 1024 * 8 * 256 - 16), None) == 5
    assert red(1, 1024, 8, 2, 128, 1, vp((1 << 20) + 8), b, None) == 4    # misaligned


def test_shift_labels_validation(L):
    vp = ctypes.c_void_p
    ids, lab, cu = vp(1 << 20), vp(1 << 30), vp(1 << 24)
    f = L.ulysses_shift_labels
    assert f(1, 1024, 4, None, None, 0, 1024, -100, lab, None) == 1
    assert f(1, 1023, 4, ids, None, 0, 1023, -100, lab, None) == 2        # n % P
    assert f(1, 1024, 4, ids, None, 0, 1025, -100, lab, None) == 2        # valid_len > n
    assert f(1, 1024, 4, ids, None, 0, -1, -100, lab, None) == 2
    assert f(1, 1024, 4, ids, None, 3, 1024, -100, lab, None) == 1        # docs without cu
    assert f(2, 1024, 4, ids, None, 0, 1024, -100, vp((1 << 20) + 4096), None) == 5
    assert f(1, 1024, 4, ids, vp((1 << 30) + 64), 2, 1024, -100, lab, None) == 5  # cu inside labels


def test_projection_validation(L):
    vp = ctypes.c_void_p
    x, w, tab, q, k, v = (vp(1 << (30 + i)) for i in range(6))
    f = L.ulysses_qkv_proj_rope
    args = lambda **kw: [kw.get("B", 1), kw.get("n", 8192), kw.get("P", 4), kw.get("hidden", 2560),
                         kw.get("H", 32), kw.get("G", 8), kw.get("d", 128), x, w, tab,
                         kw.get("max_pos", 8192), None, q, k, v, None]
    assert f(*args(n=8190)) == 2                       # n % P
    assert f(*args(G=2)) == 6                          # fewer KV heads than ranks: not fused
    assert f(*args(d=64)) == 6
    assert f(*args(hidden=2500)) == 6                  # hidden % 64
    assert f(*args(max_pos=100)) == 2                  # table shorter than the sequence
    a = args()
    a[12] = vp((1 << 30) + 64)                         # q inside x
    assert f(*a) == 5
    a = args()
    a[7] = None
    assert f(*a) == 1
    g = L.ulysses_o_proj
    assert g(1, 8192, 4, 2500, 32, 128, x, w, q, None) == 6           # hidden % 256
    assert g(1, 8190, 4, 2560, 32, 128, x, w, q, None) == 2
    assert g(1, 8192, 4, 2560, 32, 128, x, w, vp((1 << 30) + 16), None) == 5
    assert L.ulysses_rope_table(0, 128, 1e6, tab, None) == 2
    assert L.ulysses_rope_table(8192, 127, 1e6, tab, None) == 2
    assert L.ulysses_rope_table(8192, 128, 0.5, tab, None) == 2
    assert L.ulysses_rope_table(8192, 128, 1e6, vp((1 << 30) + 4), None) == 4


def test_attn_desc_validation(L):
    from long_context_sequence_all_b200 import ulysses as U
    n = ctypes.c_size_t(0)
    ok = U.make_desc(1, 8192, 4, 32, 8, 128, U.ULY_BF16, U.MASK_CAUSAL)
    assert L.ulysses_attn_bwd_workspace_size(ctypes.byref(ok), ctypes.byref(n)) == 0
    assert n.value >= 8192 * 32 * 4
    bad = [U.make_desc(1, 8190, 4, 32, 8, 128, U.ULY_BF16, 1),   # n % P
           U.make_desc(1, 8192, 4, 30, 8, 128, U.ULY_BF16, 1),   # H % P
           U.make_desc(1, 8192, 4, 32, 6, 128, U.ULY_BF16, 1),   # G % P, H % G
           U.make_desc(1, 8192, 4, 32, 8, 128, 7, 1)]            # dtype
    codes = [L.ulysses_attn_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) for d in bad]
    assert codes == [2, 2, 2, 3]
    assert L.ulysses_attn_bwd_workspace_size(
        ctypes.byref(U.make_desc(1, 8192, 4, 32, 8, 64, U.ULY_BF16, 1)), ctypes.byref(n)) == 6
    assert L.ulysses_attn_bwd_workspace_size(
        ctypes.byref(U.make_desc(1, 8192, 4, 32, 8, 128, U.ULY_BF16, 2)), ctypes.byref(n)) == 1  # no cu
    d = U.make_desc(1, 8192, 4, 32, 8, 128, U.ULY_BF16, 1)
    vp = ctypes.c_void_p
    assert L.ulysses_attn_fwd(ctypes.byref(d), None, vp(1 << 20), vp(1 << 21), vp(1 << 22),
                              vp(1 << 23), None) == 1
    # bwd without workspace
    assert L.ulysses_attn_bwd(ctypes.byref(d), *[vp(1 << (20 + i)) for i in range(9)], None, 0, None) == 10


def test_attn_desc_flags_and_workspace_sizes(L):
    """out_seq_layout and deterministic take 0 or 1.  The bf16 workspace holds
    D and LSE log2(e) per query row (n rounded up to 128 per head); the fused
    backward adds its fp32 dQ accumulator (512 bytes per padded query row)
    after a 256-byte boundary."""
    from long_context_sequence_all_b200 import ulysses as U
    n = ctypes.c_size_t(0)
    B, N, P, H, G = 1, 8000, 4, 32, 8
    rows_pad = B * H * ((N + 127) // 128 * 128)
    stats = 2 * 4 * ((rows_pad + 63) // 64 * 64)
    det = U.make_desc(B, N, P, H, G, 128, U.ULY_BF16, 1, deterministic=True)
    assert L.ulysses_attn_bwd_workspace_size(ctypes.byref(det), ctypes.byref(n)) == 0
    assert n.value == stats
    fused = U.make_desc(B, N, P, H, G, 128, U.ULY_BF16, 1, out_seq_layout=True)
    assert L.ulysses_attn_bwd_workspace_size(ctypes.byref(fused), ctypes.byref(n)) == 0
    assert n.value == (stats + 255) // 256 * 256 + rows_pad * 128 * 4
    for field in ("out_seq_layout", "deterministic"):
        bad = U.make_desc(B, N, P, H, G, 128, U.ULY_BF16, 1)
        setattr(bad, field, 2)
        assert L.ulysses_attn_bwd_workspace_size(ctypes.byref(bad), ctypes.byref(n)) == 2


def test_loss_validation(L):
    vp = ctypes.c_void_p
    n = ctypes.c_size_t(0)
    assert L.ulysses_loss_workspace_size(4, 65536, 8192, ctypes.byref(n)) == 0 and n.value > 0
    assert L.ulysses_loss_workspace_size(4, 65535, 8192, ctypes.byref(n)) == 2
    args = [vp(1 << 30), vp(1 << 20), -100, vp(1 << 21), vp(1 << 22), vp(1 << 23), vp(1 << 24), 1 << 20, None]
    assert L.ulysses_loss_aggregate(4, 1023, 8192, 1, *args) == 2
    assert L.ulysses_loss_aggregate(4, 1024, 8191, 1, *args) == 4           # row not 16 B
    assert L.ulysses_loss_aggregate(4, 1024, 8192, 9, *args) == 3
    small = args[:-3] + [vp(1 << 24), 8, None]
    assert L.ulysses_loss_aggregate(4, 1024, 8192, 1, *small) == 10


def test_library_has_no_cpu_fallback_symbols():
    """The product binding never imports the oracle."""
    src = open(os.path.join(ROOT, "long_context_sequence_all_b200", "ulysses.py")).read()
    assert "oracle" not in src.replace("no fallback", "")


def test_smoke_shape_passes_host_validation(L):
    """The shape smoke() runs on the GPU is one the library accepts (H, G
    divisible by P, H by G), so the round-end smoke cannot fail on validation."""
    import __graft_entry__ as ge
    from long_context_sequence_all_b200 import ulysses as U
    P, n, H, G, d = ge.SMOKE_SHAPE
    n_ws = ctypes.c_size_t(0)
    desc = U.make_desc(1, n, P, H, G, d, U.ULY_BF16, U.MASK_CAUSAL)
    assert L.ulysses_attn_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(n_ws)) == 0
    assert L.ulysses_loss_bwd_workspace_size(P, 256, 8192, ctypes.byref(n_ws)) == 0


def test_every_profiled_kernel_has_a_distinct_name(L):
    """The per-kernel timing table names every kernel id (an id without a
    name would make the profile unreadable)."""
    names = [L.ulysses_kernel_name(k) for k in range(L.ulysses_kernel_count())]
    assert all(n for n in names), names
    names = [n.decode() for n in names]
    assert len(set(names)) == len(names) and "unknown" not in names
    for k in ("attn_fwd_sm100", "attn_dkdv_sm100", "attn_dq_sm100", "seq_to_head", "head_to_seq",
              "loss_partial", "qkv_proj_sm100", "o_proj_sm100", "kv_seq_to_head_rep", "shift_labels"):
        assert k in names
    assert L.ulysses_kernel_name(L.ulysses_kernel_count()) == b"unknown"


def test_loss_gradient_validation(L):
    vp = ctypes.c_void_p
    T, V, P = 1024, 8192, 4
    n = ctypes.c_size_t(0)
    assert L.ulysses_loss_bwd_workspace_size(P, T, V, ctypes.byref(n)) == 0 and n.value > 0
    need = n.value
    z, y, dz = vp(1 << 32), vp(1 << 30), vp(1 << 34)           # logits 16 MiB, labels, dlogits
    S, C, Lo, ws = vp(1 << 24), vp((1 << 24) + 4096), vp((1 << 24) + 8192), vp(1 << 26)
    f = L.ulysses_loss_aggregate_bwd
    ok = [P, T, V, 1, z, y, -100, dz, S, C, Lo, ws, need, None]
    bad = list(ok); bad[7] = None
    assert f(*bad) == 1                                          # no dlogits
    bad = list(ok); bad[12] = need - 16
    assert f(*bad) == 10                                         # workspace too small
    bad = list(ok); bad[7] = vp((1 << 32) + 1024)
    assert f(*bad) == 5                                          # dlogits inside the logits
    bad = list(ok); bad[11] = vp((1 << 34) + 4096)
    assert f(*bad) == 5                                          # workspace inside dlogits
    bad = list(ok); bad[7] = vp((1 << 34) + 8)
    assert f(*bad) == 4                                          # misaligned dlogits
    bad = list(ok); bad[1] = T - 1
    assert f(*bad) == 2                                          # tokens % P


def test_error_word_null_argument(L):
    assert L.ulysses_error_word(None) == 1


def test_attn_block_order_setter_validates(L):
    """ulysses_set_attn_block_order takes the three ULY_BLOCK_ORDER_* values
    and rejects anything else with ULY_ERR_SHAPE (no device work)."""
    try:
        for order in (1, 2, 0):
            assert L.ulysses_set_attn_block_order(order) == 0
        for bad in (-1, 3, 100):
            assert L.ulysses_set_attn_block_order(bad) == 2
    finally:
        L.ulysses_set_attn_block_order(0)


def _no_launch(L, fn, want, *args):
    """A refused call: its status, and no kernel launched."""
    before = L.ulysses_launch_count()
    got = fn(*args)
    assert got == want, (got, want)
    assert L.ulysses_launch_count() == before


def test_linear_validation(L):
    vp = ctypes.c_void_p
    x, w, b, r, y, pre, ws = (vp(1 << (30 + i)) for i in range(7))
    n = ctypes.c_size_t(0)
    f, size = L.ulysses_linear, L.ulysses_linear_workspace_size
    args = lambda **k: [k.get("T", 1000), k.get("K", 512), k.get("N", 256), k.get("act", 0), k.get("x", x),
                        k.get("w", w), k.get("b", b), k.get("r", r), k.get("y", y), k.get("pre", pre),
                        k.get("ws", ws), k.get("wsb", 1 << 30), None]
    for want, kw in ((2, dict(T=-1)), (2, dict(K=0)), (4, dict(K=510)), (4, dict(N=252)), (6, dict(act=4)),
                     (6, dict(act=-1)), (1, dict(x=None)), (1, dict(w=None)), (1, dict(y=None)),
                     (4, dict(x=vp((1 << 30) + 8))), (4, dict(b=vp((1 << 32) + 2))), (5, dict(y=x)), (5, dict(y=w)),
                     (5, dict(y=vp((1 << 33) + 512))),          # partly the residual
                     (5, dict(pre=y)), (5, dict(pre=r)), (5, dict(pre=b)), (2, dict(T=1 << 40)),
                     (2, dict(T=(1 << 31) - 8192, N=1 << 20))):
        _no_launch(L, f, want, *args(**kw))
    assert f(*args(T=0, x=None, y=None)) == 0                   # no tokens: nothing to do
    assert size(1, 2560, 1024, 0, ctypes.byref(n)) == 0 and n.value == 0    # few tokens need none
    cut = dict(T=2300, K=8192, N=2304)                          # 81 tiles: 7 of them cut along K
    assert size(2300, 8192, 2304, 0, ctypes.byref(n)) == 0 and n.value > 0
    _no_launch(L, f, 10, *args(**cut, ws=None))
    _no_launch(L, f, 10, *args(**cut, wsb=n.value - 1))
    _no_launch(L, f, 5, *args(**cut, ws=x))
    assert size(1, 2560, 1024, 0, None) == 1 and size(1, 2561, 1024, 0, ctypes.byref(n)) == 4
    g = L.ulysses_linear_bwd
    dy, dx, dw, db = r, y, pre, vp(1 << 40)
    bargs = lambda **k: [k.get("T", 1000), 512, 256, k.get("act", 2), k.get("x", x), k.get("w", w), k.get("pre", b),
                         k.get("dy", dy), k.get("dx", dx), k.get("dw", dw), k.get("dt", 0), k.get("db", db),
                         k.get("ws", ws), k.get("wsb", 1 << 30), None]
    for want, kw in ((1, dict(dx=None, dw=None, db=None)), (3, dict(dt=2)), (1, dict(dy=None)), (1, dict(x=None)),
                     (1, dict(w=None)), (1, dict(pre=None)), (10, dict(ws=None)), (10, dict(wsb=64)),
                     (4, dict(dw=vp((1 << 35) + 4))), (5, dict(dx=x)), (5, dict(dx=dy)), (5, dict(dw=b)),
                     (5, dict(db=dw)), (5, dict(ws=dx))):
        _no_launch(L, g, want, *bargs(**kw))


def test_residual_norm_validation(L):
    vp = ctypes.c_void_p
    x, h, gt, wp, wq, r, u, ws = (vp(1 << (30 + i)) for i in range(8))
    nan, inf = float("nan"), float("inf")
    f = L.ulysses_residual_norm
    args = lambda **k: [k.get("B", 2), k.get("n", 512), k.get("P", 4), k.get("D", 256), k.get("dt", 1),
                        k.get("x", x), k.get("h", h), k.get("g", gt), k.get("mode", 1), k.get("wp", wp),
                        k.get("wq", wq), k.get("a", 1.0), k.get("eps", 1e-6), k.get("r", r), k.get("u", u), None]
    for want, kw in ((2, dict(B=0)), (2, dict(n=510)), (2, dict(P=0)), (2, dict(D=0)), (3, dict(dt=5)),
                     (4, dict(D=260)), (4, dict(D=258, dt=0)), (6, dict(D=16392)), (6, dict(D=8196, dt=0)),
                     (6, dict(mode=4)), (2, dict(eps=-1e-6)), (2, dict(eps=nan)), (2, dict(eps=inf)),
                     (2, dict(a=nan)), (1, dict(x=None)), (1, dict(r=None, u=None)), (1, dict(wq=None)),
                     (1, dict(g=None)), (1, dict(h=None)), (1, dict(h=None, mode=0)),
                     (4, dict(x=vp((1 << 30) + 4))), (5, dict(u=x)), (5, dict(r=gt)), (5, dict(u=r)),
                     (5, dict(r=vp((1 << 30) + 512)))):
        _no_launch(L, f, want, *args(**kw))
    g = L.ulysses_residual_norm_bwd
    n = ctypes.c_size_t(0)
    assert L.ulysses_residual_norm_bwd_workspace_size(2, 512, 256, 1, 1, ctypes.byref(n)) == 0 and n.value > 0
    dr, du, dx, dh, dwp, dwq, dg = (vp(1 << (38 + i)) for i in range(7))
    bargs = lambda **k: [2, 512, 4, 256, 1, k.get("r", r), k.get("h", h), k.get("dr", dr), k.get("du", du),
                         k.get("g", gt), k.get("mode", 1), k.get("wp", wp), k.get("wq", wq), 1.0, 1e-6,
                         k.get("dx", dx), k.get("dh", dh), k.get("dwp", dwp), k.get("dwq", dwq), k.get("dg", dg),
                         k.get("ws", ws), k.get("wsb", n.value), None]
    for want, kw in ((1, dict(dr=None, du=None)), (1, dict(r=None)), (1, dict(wq=None)), (1, dict(h=None)),
                     (1, dict(wp=None)), (1, dict(du=None)), (1, dict(mode=0)), (10, dict(ws=None)),
                     (10, dict(wsb=n.value - 1)), (5, dict(dx=du)), (5, dict(dh=dr)), (5, dict(dx=h)),
                     (5, dict(dwp=dwq)), (5, dict(dg=ws)),
                     (1, dict(dx=None, dh=None, dwp=None, dwq=None, dg=None))):
        _no_launch(L, g, want, *bargs(**kw))


def test_linear_loss_validation(L):
    vp = ctypes.c_void_p
    x, w, y, S, C, loss, ws, dx, dw = (vp(1 << (30 + i)) for i in range(9))
    n = ctypes.c_size_t(0)
    size = L.ulysses_linear_loss_workspace_size
    assert size(4, 1024, 256, 1001, ctypes.byref(n)) == 0 and n.value > 0
    f = L.ulysses_linear_loss
    args = lambda **k: [k.get("P", 4), k.get("T", 1024), k.get("D", 256), k.get("V", 1001), k.get("x", x),
                        k.get("w", w), k.get("y", y), -100, k.get("S", S), k.get("C", C), k.get("loss", loss),
                        k.get("ws", ws), k.get("wsb", 1 << 30), None]
    for want, kw in ((2, dict(P=0)), (2, dict(T=1023)), (2, dict(T=-4)), (2, dict(V=0)), (4, dict(D=252)),
                     (1, dict(x=None)), (1, dict(w=None)), (1, dict(y=None)), (1, dict(S=None)), (10, dict(ws=None)),
                     (10, dict(wsb=n.value - 1)), (4, dict(w=vp((1 << 31) + 2))), (5, dict(S=x)), (5, dict(ws=w)),
                     (5, dict(loss=S)), (2, dict(T=1 << 34))):
        _no_launch(L, f, want, *args(**kw))
    bsize = L.ulysses_linear_loss_bwd_workspace_size
    sizes = {}
    for piece in (0, 256, 1024, 5000):
        assert bsize(4, 1024, 256, 1001, 1, piece, ctypes.byref(n)) == 0
        sizes[piece] = n.value
    assert sizes[0] == sizes[1024] == sizes[5000] and sizes[256] < sizes[0] + 1001 * 256 * 4
    assert bsize(4, 1024, 256, 1001, 2, 0, ctypes.byref(n)) == 3
    assert bsize(4, 1024, 256, 1001, 1, -1, ctypes.byref(n)) == 2
    g = L.ulysses_linear_loss_bwd
    bargs = lambda **k: [4, 1024, 256, 1001, x, w, y, -100, k.get("dx", dx), k.get("dw", dw), k.get("dt", 1),
                         k.get("piece", 0), S, C, loss, k.get("ws", ws), k.get("wsb", 1 << 30), None]
    for want, kw in ((3, dict(dt=3)), (2, dict(piece=-1)), (1, dict(dx=None)), (1, dict(dw=None)),
                     (10, dict(wsb=sizes[0] - 1)), (5, dict(dx=x)), (5, dict(dw=w)), (5, dict(dx=dw)),
                     (4, dict(dx=vp((1 << 37) + 2)))):
        _no_launch(L, g, want, *bargs(**kw))


def test_tokenwise_binding_refuses_tensors_it_cannot_take(L):
    """The binding checks type, shape, layout and device before the library is called."""
    import torch
    from long_context_sequence_all_b200 import ulysses as U
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(16, 64, dtype=bf)
    y = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(2, 1, 3, 64, dtype=bf)

    def refused(status, fn, *a, **k):
        with pytest.raises(U.UlyssesError) as e:
            fn(*a, **k)
        assert e.value.status == status, e.value

    refused(3, U.ulysses_linear, x.float(), w)
    refused(2, U.ulysses_linear, x, torch.zeros(16, 72, dtype=bf))
    refused(2, U.ulysses_linear, x, w[:15], activation=U.ACT_SWIGLU)
    refused(6, U.ulysses_linear, torch.zeros(64, 4, dtype=bf).t(), w)
    refused(7, U.ulysses_linear, x, w)                                   # on the CPU
    refused(3, U.ulysses_linear_bwd, x, w, torch.zeros(4, 16))
    refused(2, U.ulysses_residual_norm, x)
    refused(2, U.ulysses_residual_norm, q, q, gate=q)                    # a gate without a mode
    refused(6, U.ulysses_residual_norm, q, q, gate=q, gate_mode=9)
    refused(3, U.ulysses_residual_norm, q.half())
    refused(7, U.ulysses_residual_norm, q, w_pre=None)
    refused(3, U.ulysses_linear_loss, x.float(), w, y, 1)
    refused(2, U.ulysses_linear_loss, q, w, y, 1)
    refused(7, U.ulysses_linear_loss, x, w, y, 1)


def test_tokenwise_binding_refuses_arguments_it_cannot_take(L):
    """What is no tensor, no number or no fitting output is an error before any launch, and the binding goes on."""
    import torch
    from long_context_sequence_all_b200 import ulysses as U
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(16, 64, dtype=bf)
    y = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(2, 1, 3, 64, dtype=bf)

    def refused(status, fn, *a, **k):
        for _ in range(2):
            with pytest.raises(U.UlyssesError) as e:
                fn(*a, **k)
            assert e.value.status == status, e.value

    before = L.ulysses_launch_count()
    refused(1, U.ulysses_linear, None, w)
    refused(1, U.ulysses_linear, x, None)
    refused(3, U.ulysses_linear, [1.0], w)
    refused(2, U.ulysses_linear, torch.zeros((), dtype=bf), w)
    refused(2, U.ulysses_linear, x, w, bias=torch.zeros(15, dtype=bf))
    refused(2, U.ulysses_linear, x, w, y=torch.zeros(4, 17, dtype=bf))
    refused(3, U.ulysses_linear, x, w, pre=torch.zeros(4, 16))
    refused(1, U.ulysses_linear_bwd, x, w, None)
    refused(1, U.ulysses_linear_bwd, x, w, torch.zeros(4, 16, dtype=bf), activation=U.ACT_GELU)   # without pre
    refused(3, U.ulysses_linear_bwd, x, w, torch.zeros(4, 16, dtype=bf), grad_dtype=torch.float16)
    refused(3, U.ulysses_linear_bwd, x, w, torch.zeros(4, 16, dtype=bf), dw=torch.zeros(16, 64, dtype=torch.float64))
    refused(1, U.ulysses_residual_norm, None)
    refused(1, U.ulysses_residual_norm_bwd, None)
    refused(1, U.ulysses_residual_norm, q, q, gate_mode=U.GATE_TOKEN)                            # without a gate
    refused(2, U.ulysses_residual_norm_bwd, q, dgate=q)
    refused(1, U.ulysses_linear_loss, x, w, None, 1)
    refused(2, U.ulysses_linear_loss, x, w, y, 0)
    refused(2, U.ulysses_linear_loss, x, w, y, 1 << 40)
    refused(2, U.ulysses_linear_loss, x, w, y[:3], 1)
    refused(3, U.ulysses_linear_loss, x, w, y.long(), 1)
    refused(3, U.ulysses_linear_loss_bwd, x, w, y, 1, grad_dtype=torch.int32)
    for fn, a, k in ((U.ulysses_linear, (x, w), dict(activation="gelu")),
                     (U.ulysses_residual_norm, (q, q), dict(gate_mode=None)),
                     (U.ulysses_linear_loss, (x, w, y, 1.5), {})):
        with pytest.raises(TypeError):
            fn(*a, **k)
    for k in (dict(ignore_index=1 << 70), dict(ignore_index=1 << 40)):
        with pytest.raises(OverflowError):
            U.ulysses_linear_loss(x, w, y, 1, **k)
    assert L.ulysses_launch_count() == before
